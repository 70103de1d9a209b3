"""64-bit forms of the linear-attention and 4-bit cache operators for the GPU tests, written
from the definitions in include/gdn.h (numpy, no code shared with the library)."""
import numpy as np

U_BF16 = 2.0 ** -8     # largest relative error of one rounding to bf16 (8-bit significand)
U_F32 = 2.0 ** -24


def linear_scan(q, k, v, g, cu, h0=None, scale=1.0):
    """o, final states, and the same sums over absolute values (for error bounds).
    q, k [T, Hk, D], v [T, Hv, D] float64; g [T, Hv] or [Hv]."""
    T, Hv, D = v.shape
    G, N = Hv // q.shape[1], len(cu) - 1
    g = np.broadcast_to(g, (T, Hv))
    o, oa = np.zeros((T, Hv, D)), np.zeros((T, Hv, D))
    hT, hA = np.zeros((N, Hv, D, D)), np.zeros((N, Hv, D, D))
    for n in range(N):
        S = np.zeros((Hv, D, D)) if h0 is None else h0[n].copy()
        A = np.abs(S)
        for t in range(cu[n], cu[n + 1]):
            a = np.exp(g[t])[:, None, None]
            kt, qt = np.repeat(k[t], G, 0), np.repeat(q[t], G, 0)
            S = np.where(a == 0, 0, a * S) + kt[:, :, None] * v[t][:, None, :]
            A = np.where(a == 0, 0, a * A) + np.abs(kt[:, :, None] * v[t][:, None, :])
            o[t] = scale * np.einsum("hi,hij->hj", qt, S)
            oa[t] = abs(scale) * np.einsum("hi,hij->hj", np.abs(qt), A)
        hT[n], hA[n] = S, A
    return o, hT, oa, hA


def key_order(D):
    n = np.arange(D)
    W, i, ng = n // 8, n % 8, D // 32
    return 32 * (W % ng) + 8 * (W // ng) + i


def value_order(D):
    n = np.arange(D)
    W, i = n // 8, n % 8
    return 64 * (W // 8) + 32 * (i // 4) + 4 * (W % 8) + i % 4


def rotate32(x, cos, sin, interleaved):
    """The rotation in fp32, products and sums rounded one by one; x [T, H, D] float32."""
    x = x.astype(np.float32).copy()
    half = cos.shape[-1]
    c, s = cos[:, None].astype(np.float32), sin[:, None].astype(np.float32)
    ia = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = b * c + a * s
    return x


def records(x, order):
    """The stored bytes of x [..., D] float32."""
    D = x.shape[-1]
    lead = x.shape[:-1]
    xg = x.reshape(lead + (D // 32, 32)).astype(np.float32)
    bad = np.isnan(xg).any(-1)
    xg = np.clip(np.where(np.isnan(xg), np.float32(-65504), xg), -65504, 65504).astype(np.float32)
    mn = xg.min(-1).astype(np.float16)
    mf = mn.astype(np.float32)
    sc = ((xg.max(-1) - mf) * np.float32(1.0 / 15.0)).astype(np.float16)
    sf = sc.astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(sf > 0, np.float32(1) / sf, np.float32(0)).astype(np.float32)
    u = np.clip(np.rint((xg - mf[..., None]) * inv[..., None]), 0, 15).astype(np.uint8)
    u = u.reshape(lead + (D,))[..., order]
    codes = u[..., 0::2] | (u[..., 1::2] << 4)
    sm = np.stack((np.where(bad, np.float16(0), sc).astype(np.float16), mn), -1)
    sm = sm.view(np.uint16).copy()
    sm[..., 1] = np.where(bad, 0x7fff, sm[..., 1])
    return np.concatenate((codes, sm.reshape(lead + (-1,)).view(np.uint8)), -1)


def values(rec, order):
    """float64 values of stored records."""
    D = len(order)
    codes = rec[..., :D // 2]
    u = np.empty(rec.shape[:-1] + (D,))
    u[..., order[0::2]] = codes & 15
    u[..., order[1::2]] = codes >> 4
    sm = np.ascontiguousarray(rec[..., D // 2:]).view(np.float16).astype(np.float64)
    return np.repeat(sm[..., 0::2], 32, -1) * u + np.repeat(sm[..., 1::2], 32, -1)


def gather(cache, table, L, which):
    """Records of positions 0 .. L-1: [L, Hkv, rec]."""
    page = cache.shape[3]
    pos = np.arange(L)
    return cache[table[pos // page], which, :, pos % page]


def attention(q, cache, table, kv_lens, cu, scale):
    """o, lse, and sum p |v| (for error bounds); q [T, Hq, D] float64."""
    T, Hq, D = q.shape
    Hkv = cache.shape[2]
    G = Hq // Hkv
    o, oa = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    for n in range(len(kv_lens)):
        L, m = int(kv_lens[n]), cu[n + 1] - cu[n]
        if m == 0 or L <= 0:
            continue
        k = np.repeat(values(gather(cache, table[n], L, 0), key_order(D)), G, 1)
        v = np.repeat(values(gather(cache, table[n], L, 1), value_order(D)), G, 1)
        for i in range(m):
            see = L - m + i + 1
            if see <= 0:
                continue
            t = cu[n] + i
            s = scale * np.einsum("hd,lhd->hl", q[t], k[:see])
            mx = s.max(1, keepdims=True)
            p = np.exp(s - mx)
            z = p.sum(1, keepdims=True)
            o[t] = np.einsum("hl,lhd->hd", p / z, v[:see])
            oa[t] = np.einsum("hl,lhd->hd", p / z, np.abs(v[:see]))
            lse[t] = (mx + np.log(z))[:, 0]
    return o, lse, oa
