"""Plain implementations, in 64 bits on the CPU, of the norm + rotation, the
quantised cache, the decode over it and the selection by length.  They follow
the formulas of include/bsa.h and share no code with the CUDA path."""
import math

import numpy as np
import torch


# ------------------------------------------------------------ norm + rotation

def encode(qkv, Hq, Hkv, q_weight, k_weight, eps, inv_freq, layout, positions, scale):
    """(q, k, v) head-major; every argument double (positions whole), layout "none", "half" or "pairs"."""
    B, N, _, d = qkv.shape
    out = []
    for x, w in ((qkv[:, :, :Hq], q_weight), (qkv[:, :, Hq:Hq + Hkv], k_weight)):
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
        if layout != "none":
            half = inv_freq.numel()
            pos = torch.arange(N).expand(B, N) if positions is None else positions
            t = pos.double()[:, :, None, None] * inv_freq
            c, s = torch.cos(t) * scale, torch.sin(t) * scale
            first = [2 * i if layout == "pairs" else i for i in range(half)]
            second = [2 * i + 1 if layout == "pairs" else i + half for i in range(half)]
            a, b = x[..., first], x[..., second]
            x = x.clone()
            x[..., first] = a * c - b * s
            x[..., second] = a * s + b * c
        out.append(x.transpose(1, 2))
    out.append(qkv[:, :, Hq + Hkv:].transpose(1, 2))
    return out


def encode_grad(qkv, Hq, Hkv, q_weight, k_weight, eps, inv_freq, layout, positions, scale, dq, dk, dv):
    """The formula's gradients (d_qkv, d_q_weight, d_k_weight) and, for error bounds, the sizes of what is summed:
    (per-row bound of d_qkv's terms, sum of |terms| of each weight's gradient)."""
    B, N, _, d = qkv.shape
    dx, dw, size, dw_size = [], [], [], []
    for x, w, dz in ((qkv[:, :, :Hq], q_weight, dq), (qkv[:, :, Hq:Hq + Hkv], k_weight, dk)):
        dy = dz.transpose(1, 2).clone()
        top = dy.abs().amax(-1, keepdim=True) * 2 * abs(scale)
        if layout != "none":
            half = inv_freq.numel()
            pos = torch.arange(N).expand(B, N) if positions is None else positions
            t = pos.double()[:, :, None, None] * inv_freq
            c, s = torch.cos(t) * scale, torch.sin(t) * scale
            first = [2 * i if layout == "pairs" else i for i in range(half)]
            second = [2 * i + 1 if layout == "pairs" else i + half for i in range(half)]
            a, b = dy[..., first], dy[..., second]
            turned = dy.clone()
            turned[..., first] = a * c + b * s
            turned[..., second] = b * c - a * s
            dy = turned
        if w is not None:
            r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
            dw.append((dy * x * r).sum((0, 1, 2)))
            dw_size.append((top * x.abs() * r).sum((0, 1, 2)))
            g = dy * w
            dx.append(r * (g - x * r * r * (g * x).mean(-1, keepdim=True)))
            big = top * w.abs().max()
            size.append(r * (big + x.abs() * r * r * (big * x.abs()).mean(-1, keepdim=True)))
        else:
            dx.append(dy)
            size.append(top.expand_as(dy))
    dx.append(dv.transpose(1, 2))
    size.append(torch.zeros_like(dx[-1]))
    return (torch.cat(dx, 2), *(dw or (None, None))), (torch.cat(size, 2), dw_size)


# ------------------------------------------------------------ quantised cache

def _e4m3_values():
    """Value of every code: sign, 4 exponent bits (bias 7), 3 fraction bits; no infinity, 0x7F and 0xFF are NaN."""
    v = np.empty(256)
    for code in range(256):
        e, f = (code >> 3) & 15, code & 7
        m = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[code] = math.nan if (code & 127) == 127 else (-m if code & 128 else m)
    return v


E4M3 = _e4m3_values()


def quantise(x):
    """(codes, exponent bytes) of rows x [..., d] float64 holding bf16 or fp32 values."""
    x = np.asarray(x, np.float64)
    flat = x.reshape(-1, x.shape[-1])
    codes, exps = np.zeros(flat.shape, np.uint8), np.zeros(len(flat), np.uint8)
    order = E4M3[:127]                      # the non-negative values, ascending
    middle = (order[1:] + order[:-1]) / 2
    for i, row in enumerate(flat):
        fine = np.isfinite(row)
        amax = np.abs(row[fine]).max(initial=0.0)
        e = 10
        while e < 246 and amax > 448.0 * 2.0 ** (e - 127):
            e += 1
        y = np.abs(np.where(fine, row, 0.0)) / 2.0 ** (e - 127)
        at = np.searchsorted(middle, y, side="left")        # a tie goes down ...
        tie = (at < 126) & (y == middle[np.minimum(at, 125)]) & (at % 2 == 1)
        at = np.where(tie, at + 1, at)                       # ... unless the lower code is odd
        c = at | np.where(np.signbit(row), 128, 0)
        codes[i] = np.where(fine, c, 127)
        exps[i] = e
    return codes.reshape(x.shape), exps.reshape(x.shape[:-1])


def dequantise(codes, exps):
    return E4M3[codes] * 2.0 ** (exps.astype(np.float64) - 127)[..., None]


# --------------------------------------------------------------------- decode

def decode(q, k_pool, v_pool, k_exp, v_exp, table, lens, idx, scale):
    """o [B,Hq,d], lse [B,Hq], and for error bounds sum p |v| and the largest sum |q k| scale of each row.
    idx None: every block."""
    q = np.asarray(q, np.float64)
    B, Hq, d = q.shape
    Hkv = k_pool.shape[1]
    G = Hq // Hkv
    o, lse = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf)
    weight, size = np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b in range(B):
        for g in range(Hkv):
            ks, vs = [], []
            blocks = range(-(-int(lens[b]) // 64)) if idx is None else [j for j in idx[b, g] if j >= 0]
            for j in blocks:
                n = min(64, int(lens[b]) - 64 * j)
                if n <= 0:
                    continue
                p = table[b, j]
                ks.append(dequantise(k_pool[p, g, :n], k_exp[p, g, :n]))
                vs.append(dequantise(v_pool[p, g, :n], v_exp[p, g, :n]))
            if not ks:
                continue
            k, v = np.concatenate(ks), np.concatenate(vs)
            for h in range(g * G, (g + 1) * G):
                x = k @ q[b, h] * scale
                top = x.max()
                p = np.exp(x - top)
                lse[b, h] = top + np.log(p.sum())
                o[b, h] = p @ v / p.sum()
                weight[b, h] = p @ np.abs(v) / p.sum()
                size[b, h] = (np.abs(k) @ np.abs(q[b, h])).max() * scale
    return o, lse, weight, size


def select(scores, lens, rows_per_len, block, kb, stride):
    """(kept lists, counts): each row's best kb of the blocks before its sequence's last, and that one."""
    rows, ncols = scores.shape
    idx, count = np.full((rows, stride), -1, np.int32), np.zeros(rows, np.int32)
    for r in range(rows):
        n = min(-(-max(int(lens[r // rows_per_len]), 0) // block), ncols)
        if n == 0:
            continue
        key = [(-np.inf, 0) if np.isnan(s) else (s, 1) for s in scores[r, :n - 1]]
        best = sorted(range(n - 1), key=lambda j: (-key[j][1], -key[j][0], j))[:kb]
        kept = sorted(best) + [n - 1]
        idx[r, :len(kept)] = kept
        count[r] = len(kept)
    return idx, count
