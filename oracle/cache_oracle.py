"""Plain float64 oracle of the paged key/value cache and of the window with visible first tokens
(numpy, CPU only, test infrastructure; shares no code with the CUDA path).

The cache itself is modelled as what each (sequence, position) holds; the byte layout is written
out separately (`row_bytes_of`) so that a test can compare whole pages."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0**-9 for m in range(8)]
                + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def to_bf16(x):
    """float64 -> float32 -> bf16 (nearest even), as float64."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    out = r.astype(np.uint32).view(np.float32).astype(np.float64)
    return np.where(np.isnan(x), np.nan, out)


def rotate(x, pos, inv_freq, mode):
    """x [..., D] at position pos (scalar), its last 2 * len(inv_freq) dims rotated, in bf16."""
    x = np.array(x, dtype=np.float64)
    if mode == "off":
        return x
    J = len(inv_freq)
    r0 = x.shape[-1] - 2 * J
    for j in range(J):
        i0, i1 = (r0 + 2 * j, r0 + 2 * j + 1) if mode == "interleaved" else (r0 + j, r0 + J + j)
        a = float(pos) * float(np.float32(inv_freq[j]))
        u, w = x[..., i0].copy(), x[..., i1].copy()
        x[..., i0] = to_bf16(u * np.cos(a) - w * np.sin(a))
        x[..., i1] = to_bf16(w * np.cos(a) + u * np.sin(a))
    return x


def _nearest_even(v, table):
    """Index of the table value nearest to each v >= 0 (ties to the even index, saturating)."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    a, b = v - table[lo], table[hi] - v
    return np.where((b < a) | ((b == a) & (hi % 2 == 0)), hi, lo)


def encode(x, tensor_scale):
    """x [..., D] -> (codes [..., D] 0..15, scales [..., D/16] e4m3 bytes).  A group with a NaN or an
    infinity has a NaN scale; a quotient past float32's range saturates."""
    with np.errstate(over="ignore"):
        y = np.asarray(x).astype(np.float32) / np.float32(tensor_scale)
    y = y.reshape(*x.shape[:-1], -1, 16)
    bad = ~np.isfinite(np.asarray(x)).reshape(y.shape).all(-1)
    y = np.where(bad[..., None], np.float32(0), y)
    s8 = _nearest_even((np.abs(y).max(-1) / np.float32(6)).astype(np.float64), E4M3)
    s = E4M3[s8].astype(np.float32)[..., None]
    z = np.divide(y, s, out=np.zeros_like(y), where=s > 0)
    code = _nearest_even(np.abs(z).astype(np.float64), E2M1) + 8 * np.signbit(z)
    s8 = np.where(bad, 0x7F, s8)
    return code.reshape(x.shape).astype(np.uint8), s8.astype(np.uint8)


def decode(codes, scales, tensor_scale):
    v = E2M1[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    s = np.where((scales & 0x7F) == 0x7F, np.nan, E4M3[np.minimum(scales & 0x7F, 126)])
    return v * np.repeat(s, 16, -1) * tensor_scale


def row_of(k, v, fmt, k_scale, v_scale):
    """(bytes of the row, k as held, v as held) of one token, k [HKV, DQK], v [HKV, DV]."""
    if fmt == "bf16":
        x = np.concatenate([k.ravel(), v.ravel()]).astype(np.float32)
        return (x.view(np.uint32) >> 16).astype(np.uint16).view(np.uint8), k, v
    (kc, ks), (vc, vs) = encode(k, k_scale), encode(v, v_scale)
    pack = lambda c: (c.reshape(-1, 2)[:, 0] | (c.reshape(-1, 2)[:, 1] << 4)).astype(np.uint8)  # noqa: E731
    row = np.concatenate([pack(kc), pack(vc), ks.ravel(), vs.ravel()])
    row = np.pad(row, (0, -len(row) % 16))
    return row, decode(kc, ks, k_scale), decode(vc, vs, v_scale)


def attend(q, k, v, keys, sm_scale, gate=None, gate_mode="sigmoid"):
    """q [H, DQK] over the keys (a list of indices into k [T, HKV, DQK], v [T, HKV, DV]).  Returns
    (out [H, DV], sum of p |v| [H, DV]), both gated."""
    H, HKV = q.shape[0], k.shape[1]
    out, mag = np.zeros((H, v.shape[2])), np.zeros((H, v.shape[2]))
    for h in range(H):
        if len(keys):
            kv = h // (H // HKV)
            s = k[keys, kv] @ q[h] * sm_scale
            p = np.exp(s - s.max())
            p /= p.sum()
            out[h], mag[h] = p @ v[keys, kv], p @ np.abs(v[keys, kv])
        if gate is not None:
            sg = 1.0 / (1.0 + np.exp(-gate[h]))
            f = sg * gate[h] if gate_mode == "silu" else sg
            out[h] *= f
            mag[h] *= abs(f)
    return out, mag


def window_keys(pos, window, n_first):
    """Keys a token at pos sees: the window and the first tokens (window 0: all)."""
    return [t for t in range(pos + 1) if window == 0 or t > pos - window or t < n_first]
