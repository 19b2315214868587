"""64-bit definitions of the operators around a paged key/value cache, in numpy,
request by request and key by key: slot maps, the rotary table and rotation,
and attention over a shared prefix followed by a request's own pages."""
from __future__ import annotations

import numpy as np


def slots(cached, new, free, table, block_size, T_cap, first_pos=0):
    """(cu_new, kv_lens, table, positions, slots, taken) from request lengths."""
    table = np.array(table, dtype=np.int64)
    P = block_size
    cu, kv, pos_out, slot_out, taken = [0], [], [], [], 0
    for r, (c, n) in enumerate(zip(cached, new)):
        c, n = max(int(c), 0), max(int(n), 0)
        for col in range(-(-c // P), -(-(c + n) // P)):
            page = free[taken] if taken < len(free) else -1
            if col < table.shape[1]:
                table[r, col] = page
            taken += 1
        for pos in range(c, c + n):
            page = table[r, pos // P] if pos // P < table.shape[1] else -1
            pos_out.append(first_pos + pos)
            slot_out.append(page * P + pos % P if page >= 0 else -1)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    pad = max(T_cap - len(pos_out), 0)
    return (np.array(cu), np.array(kv), table, np.array((pos_out + [0] * pad)[:T_cap], dtype=np.int64),
            np.array((slot_out + [-1] * pad)[:T_cap], dtype=np.int64), taken)


def rope_table(rot, first, count, base=10000.0, scaling="none", factor=1.0, context=0.0, slow=1.0, fast=32.0, attn_factor=0.0):
    """[count][rot]: cos of the rot/2 angles, then their sin, times the attention factor."""
    d = np.arange(rot // 2, dtype=np.float64)
    gain = 1.0
    f = np.power(base * (factor ** (rot / (rot - 2.0)) if scaling == "ntk" else 1.0), -2.0 * d / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        g = np.clip((context * f / (2 * np.pi) - slow) / (fast - slow), 0, 1)
        f = f * g + f / factor * (1 - g)
        gain = attn_factor if attn_factor > 0 else 0.1 * np.log(factor) + 1.0
    ang = np.arange(first, first + count, dtype=np.float64)[:, None] * f[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1) * gain


def rope(x, table_rows, rot, interleaved):
    """x [T][heads][D] turned by the table row of each token."""
    x = np.array(x, dtype=np.float64)
    c, s = np.asarray(table_rows, dtype=np.float64)[:, None, : rot // 2], np.asarray(table_rows, dtype=np.float64)[:, None, rot // 2:]
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = xa * c - xb * s, xb * c + xa * s
    return x


def attention(q, k_of, v_of, prefix_len, kv_lens, cu, scale, softcap=0.0):
    """q [T][Hq][D]; k_of(r), v_of(r): [prefix + own keys of r][Hk][D].  Returns
    out, lse, and per row what its error bound is made of: sum p |v|, the largest
    sum |q k| over the seen keys, the seen keys' number and their largest |v|."""
    T, Hq, D = q.shape
    out = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    mass, qk, seen, vmax = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq)), np.zeros((T, Hq))
    for r in range(len(kv_lens)):
        t0, t1 = int(cu[r]), int(cu[r + 1])
        if t1 <= t0:
            continue
        k, v = k_of(r), v_of(r)
        G = Hq // k.shape[1]
        for t in range(t0, t1):
            n = prefix_len + max(int(kv_lens[r]) - (t1 - t0) + (t - t0) + 1, 0)
            if n == 0:
                continue
            kk, vv = k[:n].transpose(1, 0, 2), v[:n].transpose(1, 0, 2)          # [Hk][n][D]
            qq = q[t].reshape(-1, G, D).astype(np.float64)
            with np.errstate(invalid="ignore", over="ignore"):
                s = np.matmul(qq, kk.transpose(0, 2, 1)) * scale
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                m = s.max(-1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(-1, keepdims=True)
                o = np.matmul(p / l, vv)
                out[t] = o.reshape(Hq, D)
                lse[t] = (m + np.log(l)).reshape(Hq)
                mass[t] = np.matmul(p / l, np.abs(vv)).reshape(Hq, D)
                qk[t] = np.matmul(np.abs(qq), np.abs(kk).transpose(0, 2, 1)).max(-1).reshape(Hq) * scale
                vmax[t] = np.repeat(np.abs(vv).max((1, 2)), G)
            seen[t] = n
    return out, lse, (mass, qk, seen, vmax)
