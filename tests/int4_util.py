"""64-bit oracle of the 4-bit cache, written from its definition in include/tq.h:
numpy only, no code shared with the library.

Attention tolerance (attend_bound).  With every value exact but the kernel's
arithmetic, a score is off by at most eps_s = 2^-19 S, S = the largest scale
sum_j |q_j| (|zero| + |scale c|) of the row's tokens: the queries carry 22 bits
(2^-22) and at most 24 fp32 additions or tensor-core steps of one unit in 2^-23
follow (24 2^-23 + 2^-22 < 2^-18.3; half of it on average is under 2^-19, and S
itself is a bound that signed terms stay far below).  A weight is then off by a
factor of at most 1 + 2 eps_s relative to the sum, and by the exponential and the
22-bit limbs (2^-21) and the fp32 sums (at most 2^-19), so an output is off by
V (2 eps_s + 2^-18), V = the largest |value|, plus half a step of its type.

bf16 outputs take rounded weights (`bf16`): with up to 8 query rows per kv head the
products p vs of weight and value scale are fp16 numbers, off by half a step, 2^-11
of themselves, so the output is off by at most 2^-11 times the largest code part
15 vs <= max v - min v <= 2 V of its tokens: 2^-10 V.  With more rows P and V are
rounded to fp16: 2 2^-11 V, the same; and K is too, so eps_s grows by 2^-11 S
(`rounded`)."""
import numpy as np

F15 = np.float32(0.06666667014360428)


def swizzle(d, tau):
    return 16 * ((tau & 2 if d >= 128 else 0) + (4 * (tau & 1) if d == 256 else 0))


def quantise(x, group):
    """x float32 [N, d] -> codes int [N, d], scale, zero float16 [N, d/group]."""
    n, d = x.shape
    with np.errstate(all="ignore"):
        g = np.clip(x.astype(np.float32), np.float32(-65504), np.float32(65504)).reshape(n, d // group, group)
        zero = g.min(-1).astype(np.float16)
        scale = ((g.max(-1) - zero.astype(np.float32)) * F15).astype(np.float16)
        s = scale.astype(np.float32)
        r = np.where(s > 0, np.float32(1) / s, np.float32(0)).astype(np.float32)
        t = ((g - zero.astype(np.float32)[..., None]) * r[..., None]).astype(np.float32)
        codes = np.clip(np.rint(np.nan_to_num(t, nan=0.0)), 0, 15).astype(np.int64)
    return codes.reshape(n, d), scale, zero


def values(codes, scale, zero, group):
    """float64 values the codes stand for."""
    rep = lambda v: np.repeat(v.astype(np.float64), group, axis=-1)  # noqa: E731
    return rep(zero) + rep(scale) * codes


def grid(x, group):
    """x float32 [..., d] -> the float64 values its 4-bit form stands for."""
    f = x.reshape(-1, x.shape[-1])
    return values(*quantise(f, group), group).reshape(x.shape)


def read_cache(raw, d, group, blocks, T):
    """Tokens [0, T) from packed bytes: raw uint8 [pool, block bytes], blocks: pool block of each logical block.
    Returns codes [T, d], scale, zero [T, d/group]."""
    codes = np.zeros((T, d), np.int64)
    pairs = np.zeros((T, d // group, 2), np.float16)
    for t in range(T):
        blk, tau = raw[blocks[t // 64]], t % 64
        rec = blk[tau * (d // 2):(tau + 1) * (d // 2)]
        byte = rec[np.arange(d // 2) ^ swizzle(d, tau)]
        codes[t, 0::2], codes[t, 1::2] = byte & 15, byte >> 4
        at = 64 * (d // 2) + tau * 4 * (d // group)
        pairs[t] = blk[at:at + 4 * (d // group)].view(np.float16).reshape(d // group, 2)
    return codes, pairs[..., 0], pairs[..., 1]


def attend(q, k, v, scale, n_q, every=None):
    """q [Lq, d], k, v [T, d] float64; query i sees tokens [0, T - Lq + 1 + i).  Returns [Lq, d] (every: only
    each every-th query)."""
    T = len(k)
    out = np.zeros(q.shape)
    for i in range(n_q):
        n = T - n_q + 1 + i
        if n <= 0 or (every and i % every):
            continue
        s = scale * (k[:n] @ q[i])
        p = np.exp(s - s.max())
        out[i] = (p @ v[:n]) / p.sum()
    return out


def attend_bound(q, kabs, v, scale, out, half_step, bf16=False, rounded=False):
    """Largest allowed |error| of the outputs [Lq, d]; kabs [T, d]: |zero| + |scale c|."""
    if len(v) == 0:
        return np.zeros_like(out)
    S = abs(scale) * (np.abs(q) @ kabs.T).max(-1, keepdims=True)
    eps_s = S * (2.0 ** -19 + (2.0 ** -11 if rounded else 0.0))
    return np.abs(v).max() * (2 * eps_s + 2.0 ** -18 + (2.0 ** -10 if bf16 else 0.0)) + half_step * np.abs(out) + 1e-30
