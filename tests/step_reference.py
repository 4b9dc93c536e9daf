"""fp64 references of the serving-step operators, from their definitions, and
the error bounds that the tests allow.

Bounds.  Half a step of a type, relative to the value, is u = eps / 2: bf16
2^-8, f16 2^-11, fp32 2^-24, e4m3 2^-4 (2^-10 absolute below its normal range).

Attention (weights w summing to 1, o = sum w v, A = sum w |v - o|):
  * the bf16 kernels round each weight to bf16 for the PV product and divide
    by the sum of the rounded weights: with |e| <= 2^-8,
      o' - o = sum w e (v - o) / sum w (1 + e), at most 2^-8 / (1 - 2^-8) A;
  * the e4m3 kernels pack weights as f16 and divide by the unrounded sum:
      at most 2^-11 sum w |v|, plus 2^-25 max |v| per token where a weight is
      below f16's normal range (weights are relative to a reference max whose
      own token has weight >= 1);
  * a logit is a d-term fp32 dot product: off by at most X = (d + 8) 2^-24
    scale sum |q k|, which changes o by at most 2 X A (exp within 1 + 2 X for
    small X, the same argument as for e above); ex2 and the sums add 2^-18 A;
  * rounding the output: 2^-8 |o|.
  LSE: X, plus 2^-20 (1 + |lse|) for exp2, log2, the sum and the conversions.

Norm and rotation: at most 32 fp32 roundings on the way (16 in the sum of
squares, halved by the root; rsqrt within 2 ulp; three products and one fma):
2^-19 of |a cos| + |b sin|, then the rounding to the output's type.
"""

import math

import numpy as np
import torch

DEVERR = dict(BLOCK_ID=1, SLOT=2, LENGTH=8, POSITION=16, NO_BLOCKS=32)


def plan(ctx, qlen, table, free, start, bs, num_blocks, cap):
    """(query_start_loc, seq_lens, positions, slot_mapping, totals, table, error bits)."""
    table = np.array(table, np.int32)
    n, width = table.shape
    pos, slots = np.zeros(cap, np.int32), np.full(cap, -1, np.int64)
    qsl, seqs, err, at, t = [0], [], 0, max(start, 0), 0
    if start < 0:
        err |= DEVERR["LENGTH"]
    for i in range(n):
        c, m = int(ctx[i]), int(qlen[i])
        if c < 0 or m < 0:
            err |= DEVERR["LENGTH"]
        c, m = max(c, 0), max(m, 0)
        have, need = -(-c // bs), -(-(c + m) // bs)
        fresh = {}
        for b in range(have, need):
            f = at + b - have
            first = b * bs                       # the token that opens block b
            reached = t + first - c < cap
            block = -1
            if start < 0:
                pass
            elif f >= len(free):
                err |= DEVERR["NO_BLOCKS"] if reached else 0
            elif 0 <= free[f] < num_blocks:
                block = int(free[f])
            else:
                err |= DEVERR["BLOCK_ID"] if reached else 0
            if b >= width:
                err |= DEVERR["LENGTH"] if reached else 0
                block = -1
            elif reached:
                table[i, b] = block
            fresh[b] = block
        at += need - have
        for j in range(m):
            p = c + j
            b = p // bs
            if t < cap:
                if b in fresh:
                    block = fresh[b]
                elif b >= width:
                    block, err = -1, err | DEVERR["LENGTH"]
                else:
                    block = int(table[i, b])
                    if not 0 <= block < num_blocks:
                        block, err = -1, err | DEVERR["BLOCK_ID"]
                pos[t] = p
                slots[t] = -1 if block < 0 else block * bs + p % bs
            t += 1
        qsl.append(t)
        seqs.append(c + m)
    if t > cap:
        err |= DEVERR["LENGTH"]
    return (np.minimum(qsl, cap).astype(np.int32), np.array(seqs, np.int32), pos, slots,
            np.array([t, at], np.int32), table, err)


def norm_rope(x, w, eps, cos_sin, pos, interleaved):
    """(result, sum of the magnitudes that make it) of rows x [T, H, d], fp64."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    y, mag = x.copy(), np.abs(x)
    if cos_sin is not None and cos_sin.shape[1] > 0:
        r = cos_sin.shape[1]
        for k in range(r // 2):
            a, b = (2 * k, 2 * k + 1) if interleaved else (k, k + r // 2)
            c = cos_sin[pos, k].astype(np.float64)[:, None]
            s = cos_sin[pos, r // 2 + k].astype(np.float64)[:, None]
            y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
            mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
            mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def sees(p, key, window, sinks):
    return key <= p and (key > p - window or key < sinks)


def seen_by_any(ctx, seq, window, sinks):
    """Mask over [0, seq): positions that some row of [ctx, seq) sees."""
    k = np.arange(seq)
    if seq <= ctx:
        return np.zeros(seq, bool)
    return (k >= max(0, ctx - window + 1)) | (k < min(sinks, seq))


def window_attention(q, pool, table, qsl, seqs, scale, window, sinks):
    """fp64 attention on the tensors' device.  q [T, Hq, d] and pool [nb, 2,
    bs, Hkv, d] fp64 (cells that no row sees are not read).  Returns out, lse,
    and per element the A, sum w |v|, per row X / ((d + 8) 2^-24) and the
    number of visible tokens of the bounds above."""
    T, hq, d = q.shape
    bs, hkv = pool.shape[2], pool.shape[3]
    grp, dev = hq // hkv, q.device
    out = torch.zeros((T, hq, d), dtype=torch.float64, device=dev)
    A, B = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=dev)
    X = torch.zeros((T, hq), dtype=torch.float64, device=dev)
    cnt = torch.zeros(T, dtype=torch.float64, device=dev)
    for i in range(len(seqs)):
        seq, q0, q1 = int(seqs[i]), int(qsl[i]), int(qsl[i + 1])
        ctx = seq - (q1 - q0)
        key = torch.from_numpy(np.nonzero(seen_by_any(ctx, seq, window, sinks))[0]).to(dev)
        if q1 == q0 or key.numel() == 0:
            continue
        blk = torch.as_tensor(np.asarray(table[i]), device=dev).long()[key // bs]
        k, v = pool[blk, 0, key % bs], pool[blk, 1, key % bs]          # [L, Hkv, d]
        for a in range(q0, q1, 64):
            b = min(a + 64, q1)
            p = torch.arange(ctx + a - q0, ctx + b - q0, device=dev)[:, None]
            vis = (key <= p) & ((key > p - window) | (key < sinks))
            cnt[a:b] = vis.sum(-1).double()
            for h in range(hkv):
                hs = slice(h * grp, (h + 1) * grp)
                x = torch.einsum("tgd,kd->tgk", q[a:b, hs], k[:, h]) * scale
                mag = torch.einsum("tgd,kd->tgk", q[a:b, hs].abs(), k[:, h].abs()) * abs(scale)
                X[a:b, hs] = mag.masked_fill(~vis[:, None], 0).amax(-1)
                x = x.masked_fill(~vis[:, None], -math.inf)
                lse[a:b, hs] = torch.logsumexp(x, -1)
                w = torch.softmax(x, -1).masked_fill(~vis[:, None], 0)   # a row may see nothing
                o = torch.einsum("tgk,kd->tgd", w, v[:, h])
                out[a:b, hs] = o
                B[a:b, hs] = torch.einsum("tgk,kd->tgd", w, v[:, h].abs())
                for g in range(grp):
                    hh = h * grp + g
                    gap = (v[None, :, h] - o[:, g, None, :]).abs()
                    A[a:b, hh] = torch.einsum("tk,tkd->td", w[:, g], gap)
    return out, lse, A, B, X, cnt


def check_attention(got_o, got_l, ref, d, fp8, vmax, what):
    o, lse, A, B, X, cnt = ref
    got_o, got_l = got_o.double(), got_l.double()
    logit = (d + 8) * 2.0 ** -24 * X
    tol = 2.0 ** -8 * o.abs() + (2 * logit[..., None] + 2.0 ** -18) * A + 1e-30
    if fp8:
        tol = tol + 2.0 ** -11 * B * 1.01 + (2.0 ** -25 * vmax * cnt)[:, None, None]
    else:
        tol = tol + 2.0 ** -8 / (1 - 2.0 ** -8) * A
    err = (got_o - o).abs()
    assert torch.isfinite(got_o).all(), f"{what}: non-finite output"
    worst = float((err - tol).max()) if err.numel() else 0.0
    assert worst <= 0, f"{what}: output beyond its bound by {worst:.3e}"
    empty = torch.isneginf(lse)
    assert torch.equal(empty, torch.isneginf(got_l)), f"{what}: -inf pattern"
    assert (got_o[empty] == 0).all(), f"{what}: rows with nothing visible"
    live = ~empty
    ltol = logit[live] + 2.0 ** -20 * (1 + lse[live].abs())
    lerr = (got_l[live] - lse[live]).abs()
    assert (lerr <= ltol).all(), f"{what}: lse beyond its bound by {(lerr - ltol).max():.3e}"
