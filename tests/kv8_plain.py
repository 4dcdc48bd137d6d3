"""Plain implementation of the paged 8-bit KV cache for the tests, on the CPU: the append
in fp32 step by step as the definition has it (codes are compared bit for bit), the
attention in 64 bits with a bound for the kernel's own roundings."""
import torch

TOP = {torch.int8: 127.0, torch.uint8: 448.0}


def to_codes(v, dtype):
    if dtype == torch.int8:
        return v.round().clamp(-127, 127).to(torch.int8)
    return v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def values(q):
    return q.float() if q.dtype == torch.int8 else q.view(torch.float8_e4m3fn).float()


def angles(max_pos, rot, base=10000.0):
    f = base ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return a.cos().float(), a.sin().float()


def rotate(x, pos, rope):
    """x [n, h, D] fp32 at positions pos [n]; every product and sum rounded to fp32."""
    if rope is None:
        return x
    cos, sin, inter = rope
    half = cos.shape[1]
    c, s = cos[pos][:, None], sin[pos][:, None]
    y = x.clone()
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else \
        (slice(0, half), slice(half, 2 * half))
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


def append(K, V, cache, table, cu, lens, rope):
    """The cache after the append, as new CPU tensors."""
    kq, ks, vq, vs = [t.clone() for t in cache]
    T, top = kq.shape[2], torch.tensor(TOP[kq.dtype])
    for b in range(len(lens)):
        n, start = int(cu[b + 1] - cu[b]), int(lens[b] - (cu[b + 1] - cu[b]))
        rows = slice(int(cu[b]), int(cu[b + 1]))
        pos = torch.arange(start, start + n)
        k = rotate(K[rows].float(), pos, rope)
        for x, q, s in ((k, kq, ks), (V[rows].float(), vq, vs)):
            done = 0
            while done < n:
                p = start + done
                page, slot = int(table[b, p // T]), p % T
                m = min(T - slot, n - done)
                part = x[done:done + m].transpose(0, 1)  # [heads, m, D]
                fin = torch.where(part.isfinite(), part, torch.zeros(()))
                now = torch.div(fin.abs().amax((1, 2)), top).clamp(min=1e-8)
                if slot:
                    now = torch.maximum(now, s[page])
                    r = torch.div(s[page], now)[:, None, None]
                    grown = to_codes(values(q[page, :, :slot].contiguous()) * r, q.dtype)
                    keep = (now == s[page])[:, None, None]
                    q[page, :, :slot] = torch.where(keep, q[page, :, :slot], grown)
                s[page] = now
                lim = (now * top)[:, None, None]
                part = torch.where(part.isnan(), torch.zeros(()), part)
                part = torch.minimum(torch.maximum(part, -lim), lim)
                q[page, :, slot:slot + m] = to_codes(torch.div(part, now[:, None, None]), q.dtype)
                done += m
    return kq, ks, vq, vs


def attention(Q, cache, table, cu, lens, rope, scale):
    """(result, bound) in 64 bits: |kernel - result| <= bound.

    The kernel rounds the rotated query to f16 relative to its row (half a step 2^-11 of
    each element), sums D products in fp32, and rounds a weight to f16 (2^-11).  A score
    off by d changes a weight by a factor of exp(d) at most, and the sum of the weights
    likewise; exponentials and fp32 sums are covered by 2^-10 in place of 2^-11; the
    result is rounded to its type (eps / 2)."""
    kq, ks, vq, vs = cache
    T, G, D = kq.shape[2], Q.shape[1] // kq.shape[1], Q.shape[2]
    out = torch.zeros(Q.shape, dtype=torch.float64)
    tol = torch.zeros(Q.shape, dtype=torch.float64)
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        if n == 0 or L == 0:
            continue
        pages = table[b, : -(-L // T)].long()
        k, v = [(values(q[pages]).double() * s[pages].double()[..., None, None])
                .transpose(0, 1).reshape(q.shape[1], -1, D)[:, :L].repeat_interleave(G, 0)
                for q, s in ((kq, ks), (vq, vs))]
        pos = torch.arange(L - n, L)
        q = rotate(Q[cu[b]:cu[b + 1]].float(), pos.clamp(min=0), rope).double()
        q = q.transpose(0, 1)  # [heads, n, D]
        hide = torch.arange(L)[None, :] > pos[:, None]
        s = (q @ k.transpose(1, 2) * scale).masked_fill(hide, -torch.inf)
        d = q.abs() @ k.abs().transpose(1, 2) * scale * (2.0 ** -11 + (D + 16) * 2.0 ** -23)
        d = d.masked_fill(hide, 0).amax(-1, keepdim=True)
        p = torch.softmax(s, -1)
        p = torch.where(hide.all(-1)[:, None], torch.zeros((), dtype=p.dtype), p)
        o, mag = p @ v, p @ v.abs()
        bound = mag * (torch.expm1(2 * d) + 2.0 ** -10) + o.abs() * torch.finfo(Q.dtype).eps / 2
        out[cu[b]:cu[b + 1]] = o.transpose(0, 1)
        tol[cu[b]:cu[b + 1]] = bound.transpose(0, 1)
    return out, tol + 1e-30 + (6e-8 if Q.dtype == torch.float16 else 0)


def make_state(seqs, heads, kv, D, T, code, dtype, seed, extra_cols=1, rope=None):
    """A cache holding the older positions of `seqs` [(new, length)], and the new rows.
    Slots and pages nobody wrote hold 0xFF bytes and NaN scales; unused table entries
    are -1."""
    g = torch.Generator().manual_seed(seed)
    B = len(seqs)
    need = [-(-max(L, 1) // T) for _, L in seqs]
    P = sum(need) + 2
    perm = torch.randperm(P, generator=g)
    table = torch.full((B, max(need) + extra_cols), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, : need[b]] = perm[at:at + need[b]].to(torch.int32)
        at += need[b]
    cu = torch.tensor([0] + [n for n, _ in seqs]).cumsum(0).to(torch.int32)
    lens = torch.tensor([L for _, L in seqs], dtype=torch.int32)
    cache = []
    for _ in range(2):
        q = torch.full((P, kv, T, D), 255, dtype=torch.uint8).view(code)
        cache += [q, torch.full((P, kv), float("nan"))]
    for b, (n, L) in enumerate(seqs):
        for p in range(0, max(0, L - n), T):
            m, page = min(T, L - n - p), int(table[b, p // T])
            for q, s in ((cache[0], cache[1]), (cache[2], cache[3])):
                x = torch.randn(kv, m, D, generator=g) * (0.2 + 3 * torch.rand(1, generator=g))
                x[..., 3] *= 5
                s[page] = x.abs().amax((1, 2)) / TOP[code]
                q[page, :, :m] = to_codes(x / s[page][:, None, None], code)
    rows = int(cu[-1])
    qkv = torch.randn(max(rows, 1), heads + 2 * kv, D, generator=g)
    qkv[..., 5] *= 4
    qkv = qkv.to(dtype)[:rows]
    return dict(cache=tuple(cache), table=table, cu=cu, lens=lens, rope=rope,
                Q=qkv[:, :heads], K=qkv[:, heads:heads + kv], V=qkv[:, heads + kv:],
                max_new=max(1, max(n for n, _ in seqs)))


def on_gpu(st):
    d = dict(st)
    n, heads, D = st["Q"].shape
    kv = st["K"].shape[1]
    qkv = torch.cat([st["Q"], st["K"], st["V"]], 1).cuda()
    d["Q"], d["K"], d["V"] = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    d["cache"] = tuple(t.cuda() for t in st["cache"])
    for k in ("table", "cu", "lens"):
        d[k] = st[k].cuda()
    if st["rope"] is not None:
        d["rope"] = (st["rope"][0].cuda(), st["rope"][1].cuda(), st["rope"][2])
    return d
