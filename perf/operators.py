"""Measured cases of the 8-bit attention block: the block-scaled FP8 quantizer and
product (the projections), the paged 8-bit KV cache's append with rotary positions,
and the attention that reads that cache.

`run` computes each operator in its plain form (elementary torch operations in fp32)
or, where `own` is true, through this repository's entry points.  A case is a dict of
plain values; its "op" names the operator:

quant   E4M3 codes and one fp32 scale per block of `rows` x 128 elements
gemm    Y = X W^T with X [M, K] bf16 quantized per token and 128 elements, W [N, K]
        quantized per 128 x 128 block, both E4M3
append  K, V rows of `batch` sequences rotated, quantized and written into a paged
        cache with one scale per (page, head)
attn    causal attention of `new` queries per sequence over that cache
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def _quant(name, R, K, rows, dtype="bf16"):
    return {"name": name, "op": "quant", "R": R, "K": K, "rows": rows, "dtype": dtype}


def _gemm(name, M, N, K):
    return {"name": name, "op": "gemm", "M": M, "N": N, "K": K}


def _kv(name, op, batch, new, past, heads, kv, D, page, fmt, dtype="bf16", ragged=True,
        inter=False, rot=None):
    return {"name": name, "op": op, "batch": batch, "new": new, "past": past, "heads": heads,
            "kv": kv, "D": D, "page": page, "fmt": fmt, "dtype": dtype, "ragged": ragged,
            "inter": inter, "rot": D if rot is None else rot}


def listed():
    return [
        # a 70B layer's largest weight, quantized once when a model is loaded
        _quant("quant-w-28672x8192", 28672, 8192, 128),
        # one prefill batch's activations in front of a down projection
        _quant("quant-x-2048x11008", 2048, 11008, 1),
        # one token through the 70B up projection: the weight is read once
        _gemm("gemm-1x28672x8192", 1, 28672, 8192),
        # a small serving batch through the 7B down projection
        _gemm("gemm-16x4096x11008", 16, 4096, 11008),
        # a ragged prefill chunk, odd everywhere, last K block partial
        _gemm("gemm-333x11000x4112", 333, 11000, 4112),
        # a full prefill batch through the 7B up projection
        _gemm("gemm-4096x11008x4096", 4096, 11008, 4096),
        # one decode step of a serving batch: a token per sequence
        _kv("append-decode-64", "append", 64, 1, 4096, 64, 8, 128, 64, "e4m3"),
        # prompts of several requests written at once
        _kv("append-prefill-4x2048", "append", 4, 2048, 100, 64, 8, 128, 64, "int8"),
        # one short conversation: latency
        _kv("attn-decode-1x513", "attn", 1, 1, 512, 32, 8, 128, 16, "e4m3", ragged=False),
        # a serving batch's decode step, lengths from a few tokens to 8192
        _kv("attn-decode-64x8192", "attn", 64, 1, 8191, 64, 8, 128, 64, "int8"),
        # drafted tokens checked against a long context
        _kv("attn-verify-4x5x32768", "attn", 4, 5, 32763, 32, 8, 128, 64, "e4m3", "fp16"),
        # a prompt chunk behind earlier chunks
        _kv("attn-prefill-2x2048", "attn", 2, 2048, 4096, 32, 8, 128, 64, "e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "append", "attn", "attn"])
    if op == "quant":
        K = 16 * _log(rng, 1, 700)
        R = min(_log(rng, 1, 28672), 28672 * 8192 // K)
        c = _quant("", R, K, rng.choice([1, 128]), rng.choice(["bf16", "fp16", "fp32"]))
    elif op == "gemm":
        N, K = 8 * _log(rng, 16, 3584), 16 * _log(rng, 8, 700)
        K = min(K, 28672 * 8192 // N // 16 * 16)
        M = min(_log(rng, 1, 4096), 4096 * 11008 * 4096 // (N * K))
        c = _gemm("", max(1, M), N, K)
    else:
        kv, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 128, 256])
        group = rng.choice([1, 2, 3, 4, 8, 12])
        page, fmt = rng.choice([16, 32, 64, 128]), rng.choice(["int8", "e4m3"])
        dtype, inter = rng.choice(["bf16", "fp16"]), rng.random() < 0.3
        rot = D if rng.random() < 0.7 else D // 2
        if op == "append":
            new = _log(rng, 1, 2048)
            batch = max(1, min(_log(rng, 1, 64), 8192 // new))
            past = _log(rng, 1, 2048)
        else:
            new = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 1500)])
            past = _log(rng, 1, 16384)
            batch = max(1, min(_log(rng, 1, 64), 2 ** 18 // (past + new)))
            batch = max(1, min(batch, 2 ** 26 // (new * kv * group * (past + new) // 8 + 1)))
            past = min(past, max(1, 2 ** 29 // (new * kv * group * batch)))
        c = _kv("", op, batch, new, past, kv * group, kv, D, page, fmt, dtype,
                rng.random() < 0.8, inter, rot)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) & 0x7FFFFFFF)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _outliers(g, x, count, factor):
    """A few fixed channels of larger magnitude, as activations and keys have."""
    at = torch.randperm(x.shape[-1], generator=g, device=DEV)[:count]
    x[..., at] *= factor
    return x


def _lengths(case, seed):
    """New and past token counts of each sequence, in the seed's order; one sequence has
    the most of both."""
    r = random.Random(case["past"] * 7919 + case["new"])
    both = []
    for b in range(case["batch"]):
        full = b == 0 or not case["ragged"]
        both.append((case["new"] if full else r.randint((case["new"] + 1) // 2, case["new"]),
                     case["past"] if full else r.randint(0, case["past"])))
    random.Random(int(seed)).shuffle(both)
    return [n for n, _ in both], [p for _, p in both]


def _angles(case, length):
    half = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    a = torch.arange(length, dtype=torch.float64, device=DEV)[:, None] * f
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "quant":
        x = _outliers(g, _randn(g, case["R"], case["K"]), 6 if case["K"] > 64 else 1, 30.0)
        return {"case": case, "x": x.to(DT[case["dtype"]])}
    if case["op"] == "gemm":
        x = _outliers(g, _randn(g, case["M"], case["K"]), 6, 30.0).to(torch.bfloat16)
        w = _randn(g, case["N"], case["K"]).mul_(0.02).to(torch.bfloat16)
        wq, ws = _quant_plain(w, 128)
        return {"case": case, "x": x, "wq": wq, "w_scales": ws}
    new, past = _lengths(case, seed)
    B, H, D, T, kv = case["batch"], case["heads"], case["D"], case["page"], case["kv"]
    total = [n + p for n, p in zip(new, past)]
    width = -(-max(total) // T)
    need = [-(-t // T) for t in total]
    P = sum(need) + 3
    order = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    # row b of the table: its share of the shuffled pages, -1 behind the last
    first = torch.tensor([sum(need[:b]) for b in range(B)], device=DEV)[:, None]
    col = torch.arange(width, device=DEV)[None, :]
    inside = col < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(inside, order[(first + col).clamp(max=P - 1)], -1).to(torch.int32)
    cu = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device=DEV)
    lens = torch.tensor(total, dtype=torch.int32, device=DEV)
    cache = []
    for k in range(2):
        x = _randn(g, P, kv, T, D)
        x = _outliers(g, x, 4, 6.0) if k == 0 else x
        s = x.abs().amax((2, 3)) / (127.0 if case["fmt"] == "int8" else 448.0)
        cache += [_codes(x / s[:, :, None, None], case["fmt"]), s]
    cos, sin = _angles(case, max(total))
    n, dt = sum(new), DT[case["dtype"]]
    st = {"case": case, "cache": tuple(cache), "table": table, "cu": cu, "lens": lens,
          "cos": cos, "sin": sin, "max_new": max(new)}
    if case["op"] == "append":
        # keys and values are columns of one fused projection's output
        qkv = _randn(g, n, H + 2 * kv, D)
        qkv[:, H:H + kv] = _outliers(g, qkv[:, H:H + kv].clone(), 4, 6.0)
        qkv = qkv.to(dt)
        st["k"], st["v"] = qkv[:, H:H + kv], qkv[:, H + kv:]
    else:
        st["q"] = _randn(g, n, H, D).to(dt)
        if own:
            import bit_gemm_group_b200 as wq
            st["ws"] = wq.attn_kv8_workspace(B, H, kv, D, st["max_new"], DEV)
    return st


# ------------------------------------------------------------------ plain forms

def _codes(v, fmt):
    """8-bit codes of scaled values: int8, or E4M3 as uint8."""
    if fmt == "int8":
        return v.round().clamp_(-127, 127).to(torch.int8)
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(q):
    return q.float() if q.dtype == torch.int8 else q.view(torch.float8_e4m3fn).float()


def _shown(q):
    """Codes as the values they stand for (times their scale)."""
    return q.to(torch.bfloat16) if q.dtype == torch.int8 else q.view(torch.float8_e4m3fn)


def _padded(x, rows):
    R, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % 128, 0, -R % rows))


def _quant_plain(x, rows):
    R, K = x.shape
    p = _padded(x.float(), rows)
    p = p.view(p.shape[0] // rows, rows, p.shape[1] // 128, 128)
    # (a Python number as the divisor would become a multiplication by its reciprocal)
    s = p.abs().amax((1, 3))
    s = (s / s.new_full((1, 1), 448.0)).clamp(min=1e-8)
    q = _codes(p / s[:, None, :, None], "e4m3")
    return q.reshape(q.shape[0] * rows, -1)[:R, :K].contiguous(), s


def _dequant_plain(q, s, rows):
    R, K = q.shape
    w = s.repeat_interleave(128, 1)[:, :K]
    w = w.repeat_interleave(rows, 0)[:R] if rows > 1 else w
    return _values(q) * w


def _rotate(x, cos, sin, inter):
    """x [n, h, D] fp32, cos and sin [n, r / 2]: the first r elements of each head."""
    half = cos.shape[-1]
    c, s, r = cos[:, None], sin[:, None], x[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., :half], r[..., half:])
    u, v = a * c - b * s, b * c + a * s
    r = torch.stack((u, v), -1).flatten(-2) if inter else torch.cat((u, v), -1)
    return torch.cat((r, x[..., 2 * half:]), -1)


def _rows(st, n):
    """Sequence and position of each of the n new rows."""
    t = torch.arange(n, device=DEV)
    cu = st["cu"].long()
    b = torch.searchsorted(cu, t, right=True) - 1
    count = cu[1:] - cu[:-1]
    i = t - cu[b]
    return b, i, st["lens"].long()[b] - count[b] + i


def _append_plain(st):
    c = st["case"]
    T, top = c["page"], 127.0 if c["fmt"] == "int8" else 448.0
    kq, ks, vq, vs = st["cache"]
    n = st["k"].shape[0]
    b, i, pos = _rows(st, n)
    page, slot = st["table"][b, pos // T].long(), pos % T
    k = _rotate(st["k"].float(), st["cos"][pos], st["sin"][pos], c["inter"])
    # the page that each sequence's first new row falls into keeps its older rows
    cu, lens = st["cu"].long(), st["lens"].long()
    start = lens - (cu[1:] - cu[:-1])
    old = torch.gather(st["table"].long(), 1, (start // T)[:, None])[:, 0]
    kept = start % T
    for x, q, s in ((k, kq, ks), (st["v"].float(), vq, vs)):
        m = torch.zeros_like(s).index_reduce_(0, page, x.abs().amax(-1), "amax")
        before = s[old]
        new = (m / m.new_full((1, 1), top)).clamp_(min=1e-8)
        s[page] = new[page]
        grown = torch.where((kept > 0)[:, None], torch.maximum(new[old], before), new[old])
        s[old] = grown
        v = _values(q[old]) * (before / grown)[:, :, None, None]
        mine = torch.arange(T, device=DEV)[None, :] < kept[:, None]
        q[old] = torch.where(mine[:, None, :, None], _codes(v, c["fmt"]), q[old])
        q[page, :, slot] = _codes(x / s[page][:, :, None], c["fmt"])
    return [_shown(kq), ks, _shown(vq), vs]


def _attn_plain(st):
    c = st["case"]
    kq, ks, vq, vs = st["cache"]
    B, kv, D, T = c["batch"], c["kv"], c["D"], c["page"]
    G, m, width = c["heads"] // kv, st["max_new"], st["table"].shape[1]
    at = st["table"].long().clamp(min=0)

    def gather(q, s):
        x = _values(q[at]) * s[at][..., None, None]  # [B, width, kv, T, D]
        return x.transpose(1, 2).reshape(B, kv, width * T, D)

    n = st["q"].shape[0]
    b, i, pos = _rows(st, n)
    q = _rotate(st["q"].float(), st["cos"][pos], st["sin"][pos], c["inter"])
    cu, lens = st["cu"].long(), st["lens"].long()
    rows = (cu[:-1, None] + torch.arange(m, device=DEV)).clamp(max=n - 1)  # [B, m]
    q = q[rows].view(B, m, kv, G, D).permute(0, 2, 3, 1, 4).reshape(B, kv, G * m, D)
    s = (q @ gather(kq, ks).transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    last = lens[:, None] - (cu[1:] - cu[:-1])[:, None] + torch.arange(m, device=DEV)
    hide = torch.arange(width * T, device=DEV) > torch.minimum(last, lens[:, None] - 1)[..., None]
    s = s.view(B, kv, G, m, -1).masked_fill_(hide[:, None, None], -math.inf)
    s = (s - s.amax(-1, keepdim=True)).exp_()
    s = s.div_(s.sum(-1, keepdim=True)).view(B, kv, G * m, -1)
    o = (s @ gather(vq, vs)).view(B, kv, G, m, D).permute(0, 3, 1, 2, 4)  # [B, m, kv, G, D]
    return o[b, i].reshape(n, kv * G, D).to(st["q"].dtype)


def run(state):
    c, st = state["case"], state
    if not own:
        if c["op"] == "quant":
            q, s = _quant_plain(st["x"], c["rows"])
            return [_shown(q), s]
        if c["op"] == "gemm":
            q, s = _quant_plain(st["x"], 1)
            w = _dequant_plain(st["wq"], st["w_scales"], 128)
            return (_dequant_plain(q, s, 1) @ w.t()).to(torch.bfloat16)
        return _append_plain(st) if c["op"] == "append" else _attn_plain(st)
    import bit_gemm_group_b200 as wq
    if c["op"] == "quant":
        q, s = wq.quantize_fp8_block(st["x"], c["rows"])
        return [_shown(q), s]
    if c["op"] == "gemm":
        return wq.gemm_fp8_block(st["x"], st["wq"], st["w_scales"])
    rope = (st["cos"], st["sin"], c["inter"])
    if c["op"] == "append":
        wq.kv8_append(st["k"], st["v"], st["cache"], st["table"], st["cu"], st["lens"],
                      st["max_new"], rope)
        kq, ks, vq, vs = st["cache"]
        return [_shown(kq), ks, _shown(vq), vs]
    return wq.attn_kv8(st["q"], st["cache"], st["table"], st["cu"], st["lens"], st["max_new"],
                       rope=rope, ws=st["ws"])


# ------------------------------------------------------------------ 64 bits

def _e4m3_64(v):
    """The nearest E4M3 value, ties to even, saturated: steps of 2^(e - 3), e >= -6."""
    _, e = torch.frexp(v)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _code64(v, fmt):
    return torch.round(v).clamp(-127, 127) if fmt == "int8" else _e4m3_64(v)


def _blocks64(x, rows):
    """(code values, scales) of the block quantizer by its definition."""
    R, K = x.shape
    rb = torch.arange(R, device=DEV) // rows
    q = torch.empty(R, K, dtype=torch.float64, device=DEV)
    s = torch.zeros(int(rb[-1]) + 1, -(-K // 128), dtype=torch.float64, device=DEV)
    for j in range(s.shape[1]):
        part = x[:, 128 * j:128 * j + 128].double()
        a = torch.zeros(s.shape[0], dtype=torch.float64, device=DEV)
        a.scatter_reduce_(0, rb, part.abs().amax(1), "amax")
        s[:, j] = (a / 448.0).clamp(min=1e-8)
        # the code is defined by the binary32 quotient (ties of bf16 values are common)
        v = (part / s[rb, j].float().double()[:, None]).float().double()
        q[:, 128 * j:128 * j + 128] = _e4m3_64(v)
    return q, s


def _rope64(x, pos, rot, inter):
    half = rot // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
    a = (pos.double()[:, None] * f)[:, None, :]
    i = torch.arange(half, device=DEV)
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + half)
    y = x.clone()
    y[..., lo] = x[..., lo] * a.cos() - x[..., hi] * a.sin()
    y[..., hi] = x[..., hi] * a.cos() + x[..., lo] * a.sin()
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        q, s = _blocks64(st["x"], case["rows"])
        return [q, s]
    if case["op"] == "gemm":
        q, s = _blocks64(st["x"], 1)
        K = case["K"]
        y = torch.zeros(case["M"], case["N"], dtype=torch.float64, device=DEV)
        nb = torch.arange(case["N"], device=DEV) // 128
        for j in range(-(-K // 128)):
            cols = slice(128 * j, min(K, 128 * j + 128))
            w = st["wq"][:, cols].view(torch.float8_e4m3fn).double()
            y += (q[:, cols] @ w.t()) * s[:, j:j + 1] * st["w_scales"].double()[nb, j]
        return y
    T, fmt, D = case["page"], case["fmt"], case["D"]
    new, past = _lengths(case, seed)
    kq, ks, vq, vs = st["cache"]
    table = st["table"].tolist()
    if case["op"] == "append":
        top = 127.0 if fmt == "int8" else 448.0
        out = []
        for which, q, s in (("k", kq, ks), ("v", vq, vs)):
            val, sc = _values(q).double(), s.double()
            at = 0
            for b in range(case["batch"]):
                x = st[which][at:at + new[b]].double()
                pos = torch.arange(past[b], past[b] + new[b], device=DEV)
                x = _rope64(x, pos, case["rot"], case["inter"]) if which == "k" else x
                p, done = past[b], 0
                while done < new[b]:
                    page, slot = table[b][p // T], p % T
                    n = min(T - slot, new[b] - done)
                    part = x[done:done + n].transpose(0, 1)  # [kv, n, D]
                    now = (part.abs().amax((1, 2)) / top).clamp(min=1e-8)
                    if slot:
                        now = torch.maximum(now, sc[page])
                        val[page, :, :slot] = _code64(
                            val[page, :, :slot] * (sc[page] / now)[:, None, None], fmt)
                    sc[page] = now
                    val[page, :, slot:slot + n] = _code64(part / now[:, None, None], fmt)
                    p, done = p + n, done + n
                at += new[b]
            out += [val, sc]
        return out
    G, outs, at = case["heads"] // case["kv"], [], 0
    for b in range(case["batch"]):
        n, L = new[b], new[b] + past[b]
        pages = st["table"][b, :-(-L // T)].long()
        kk, vv = ((_values(q[pages]).double() * s[pages].double()[:, :, None, None])
                  .transpose(0, 1).reshape(case["kv"], -1, D)[:, :L] for q, s in ((kq, ks), (vq, vs)))
        pos = torch.arange(past[b], L, device=DEV)
        q = _rope64(st["q"][at:at + n].double(), pos, case["rot"], case["inter"])
        o = torch.empty(n, case["heads"], D, dtype=torch.float64, device=DEV)
        for h in range(case["heads"]):
            w = q[:, h] @ kk[h // G].t() / math.sqrt(D)
            w = w.masked_fill(torch.arange(L, device=DEV) > pos[:, None], -math.inf)
            o[:, h] = torch.softmax(w, -1) @ vv[h // G]
        outs.append(o)
        at += n
    return torch.cat(outs)


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "quant":
        n, size = case["R"] * case["K"], {"fp32": 4}.get(case["dtype"], 2)
        blocks = -(-case["R"] // case["rows"]) * -(-case["K"] // 128)
        return {"bytes": n * (size + 1) + 4 * blocks, "flops": 2 * n}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // 128)
        return {"bytes": N * K + 4 * kb * -(-N // 128) + 2 * M * (N + K), "flops": 2 * M * N * K}
    # ragged counts at their mean: new in [(n + 1) / 2, n], past in [0, p], the first one full
    rest = case["batch"] - 1
    mean = 0.75 if case["ragged"] and case["new"] > 1 else 1.0
    half = 0.5 if case["ragged"] else 1.0
    n = case["new"] * (1 + rest * mean)
    D, kv = case["D"], case["kv"]
    if case["op"] == "append":
        size = 4 if case["dtype"] == "fp32" else 2
        pages = n / case["page"] + case["batch"]
        return {"bytes": n * (2 * kv * D * (size + 1) + 4 * case["rot"]) + 16 * pages * kv,
                "flops": 8 * n * kv * D}
    keys = case["past"] * (1 + rest * half) + n
    pages = keys / case["page"]
    pairs = case["new"] * (case["past"] + case["new"] / 2) + \
        rest * case["new"] * mean * (case["past"] * half + case["new"] * mean / 2)
    return {"bytes": keys * 2 * kv * D + 8 * pages * kv + 4 * n * case["heads"] * D,
            "flops": 4 * pairs * case["heads"] * D}
