"""64-bit references of the chunk, read-back and windowed operators, from the cache's documented layouts (layout.py) and
the operators' formulas."""
import numpy as np

from layout import D, GpuState

HALF_BF16 = 2.0 ** -8      # half a bf16 step, relative
HALF_FP16 = 2.0 ** -11     # half an fp16 step, relative


def f16(a):
    return np.ascontiguousarray(a).view(np.float16).astype(np.float64)


def bf16(a):
    return (np.ascontiguousarray(a).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def e4m3_table():
    import torch
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)


def rotate(k, pos, theta):
    """Keys [t, D] before RoPE at positions pos [t] -> rotated."""
    ang = pos[:, None] * theta ** (-2.0 * np.arange(D // 2) / D)
    c, s = np.cos(ang), np.sin(ang)
    out = np.empty_like(k)
    out[:, 0::2] = k[:, 0::2] * c - k[:, 1::2] * s
    out[:, 1::2] = k[:, 0::2] * s + k[:, 1::2] * c
    return out


def cached_rows(st: GpuState, b: int, h: int, rope: bool = False, theta: float = 0.0):
    """k^, v^ (float64 [n, D]) of every token that unit (b, h) holds."""
    n, nq = int(st.seq_len[b]), int(st.n_quant[b])
    pad = (nq + 15) // 16 * 16
    k = np.zeros((n, D))
    v = np.zeros((n, D))
    if nq:
        u = st.unit(b, h, pad)
        if st.bits == 8:
            t = e4m3_table()
            k[:nq] = t[u["k_codes"][:nq]] * float(st.fp8_scale[0, h])
            v[:nq] = t[u["v_codes"][:nq]] * float(st.fp8_scale[1, h])
        else:
            if st.bits == 16:
                ks, kz = f16(u["k_scale"])[:, None], f16(u["k_zero"])[:, None]
            else:
                ks, kz = f16(u["k_scale"]).repeat(st.G, 0), f16(u["k_zero"]).repeat(st.G, 0)
            k[:nq] = (u["k_codes"] * ks + kz)[:nq]
            v[:nq] = (u["v_codes"] * f16(u["v_scale"])[:, None] + f16(u["v_zero"])[:, None])[:nq]
        if st.sparse:
            for g in range(nq // st.G):
                e = st.k_sparse[b, h, g]
                k[g * st.G + (e >> 16).astype(int), np.arange(D)] = bf16((e & 0xFFFF).astype(np.uint16))
            e = st.v_sparse[b, h, :nq]
            v[np.arange(nq), (e >> 16).astype(int)] = bf16((e & 0xFFFF).astype(np.uint16))
    if n > nq:
        W = st.k_ring.shape[2]
        slots = np.arange(nq, n) % W
        k[nq:], v[nq:] = bf16(st.k_ring[b, h, slots]), bf16(st.v_ring[b, h, slots])
    if rope:
        k = rotate(k, np.arange(n, dtype=np.float64), theta)
    return k, v


def visible(pos, t, window, sinks):
    see = t[None, :] <= pos[:, None]
    if window > 0:
        see &= (t[None, :] > pos[:, None] - window) | (t[None, :] < sinks)
    return see


def attend(q, k, v, pos, scale, window=0, sinks=0, present=None, rounded=True):
    """softmax(scale q k^T) v for rows q [m, D] at positions pos over keys 0..t-1; also the log-sum-exp and how far a
    kernel may be off: scores off by `d` at most change the weights by a factor within e^(2d), which moves the output by
    at most (e^(2d) - 1) sum p|v|.
      rounded: keys and values rounded to fp16 (half a step each: d grows by scale sum|q||k| 2^-11, values by 2^-11),
      weights to bf16 where the keys are bf16 (2^-8) and to fp16 elsewhere (2^-11, and 2^-25 absolute below its normal
      numbers, against a sum of weights of at least 1), out to bf16 (2^-8).
      Otherwise everything is held in 32 bits: 2^-24 per step of at most `t` steps, taken together as 2^-18."""
    t = np.arange(k.shape[0])
    see = visible(np.asarray(pos), t, window, sinks)
    if present is not None:
        see &= present[None, :]
    s = np.where(see, scale * (q @ k.T), -np.inf)
    top = s.max(1, keepdims=True) if k.shape[0] else np.full((len(q), 1), -np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(1, keepdims=True)
    p = e / np.where(total > 0, total, 1.0)
    out = p @ v
    lse = np.where(total > 0, top + np.log(np.where(total > 0, total, 1.0)), -np.inf)[:, 0]
    mag = np.where(see, abs(scale) * (np.abs(q) @ np.abs(k).T), 0.0).max(1, initial=0.0)[:, None]
    if rounded:
        d = mag * (HALF_FP16 + 2.0 ** -17) + 2.0 ** -18
        tol = (np.expm1(2 * d) + HALF_FP16 + HALF_BF16) * (p @ np.abs(v)) + HALF_BF16 * np.abs(out)
        tol += k.shape[0] * 2.0 ** -25 * np.abs(v).max(initial=0.0) + 1e-30
    else:
        d = mag * 2.0 ** -18 + 2.0 ** -18
        tol = (np.expm1(2 * d) + 2.0 ** -18) * (p @ np.abs(v)) + 1e-30
    return out, lse, tol
