"""References of the longer-context operators (4-bit pool, weight sums, eviction,
packed prompts), from their definitions; attention and its bounds are
step_reference's.

4-bit attention: code * scale is exact in f16, weights are f16 and the divisor is the
unrounded sum: step_reference's bounds for e4m3.

Weight sums: with x the logit and both in fp32, exp2(x log2(e) - lse log2(e)) is off
in its exponent by the logit's and the lse's bounds and at most 16 fp32 roundings of
magnitudes up to |x| + |lse| + 1; the sum over the heads and the addition to what was
there by (heads + 1) 2^-24 of their total.
"""

import math

import numpy as np
import torch

from tests import step_reference as ref

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BIG = 2 ** 31 - 1


def e4m3_values():
    return torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


def quantise(x, step):
    """(codes 0..15 [..., d], scale bytes [..., d / 16]) of fp32-representable x."""
    x = np.asarray(x, np.float32)
    step = np.float32(step)
    blk = x.reshape(*x.shape[:-1], -1, 16)
    nan = np.isnan(blk).any(-1)
    with np.errstate(all="ignore"):
        want = (np.abs(np.where(np.isnan(blk), 0, blk)).max(-1) / step) / np.float32(6)
        scale = torch.from_numpy(np.minimum(want, np.float32(448))).to(torch.float8_e4m3fn)
        scale = scale.view(torch.uint8).numpy().copy()
        scale[nan] = 0x7F
        s = e4m3_values()[scale].astype(np.float32)
        t = (s * step)[..., None]
        z = np.abs(blk / t)
        code = np.zeros(blk.shape, np.uint8)
        for k, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
            code += (z > m) if k % 2 == 0 else (z >= m)      # ties to the even code
        code += 8 * np.signbit(blk).astype(np.uint8)
        code = np.where(t > 0, code, 0).astype(np.uint8)     # (NaN scales too)
    return code.reshape(x.shape), scale


def fp4_parts(pool):
    """Views [nb, Hkv, groups, 2, 16, .] of a 4-bit pool's codes and scales."""
    d = pool.shape[-1] // 9
    codes = pool[..., :8 * d].reshape(*pool.shape[:-1], 16, d // 2)
    return codes, pool[..., 8 * d:].reshape(*pool.shape[:-1], 16, d // 16)


def fp4_values(pool, k_scale, v_scale):
    """The fp64 pool [nb, 2, bs, Hkv, d] that a 4-bit pool (torch uint8) stands for."""
    codes, scales = fp4_parts(pool)
    level = torch.tensor(np.concatenate([E2M1, -E2M1]), device=pool.device)
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    s = scales.contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    v = level[both] * s                                          # [nb, h, g, 2, 16, d]
    step = torch.tensor([np.float32(k_scale), np.float32(v_scale)], dtype=torch.float64,
                        device=pool.device)
    v = v * step.view(1, 1, 1, 2, 1, 1)
    nb, h, g, _, _, d = v.shape
    return v.permute(0, 3, 2, 4, 1, 5).reshape(nb, 2, g * 16, h, d)


def fp4_store(pool, which, slots, x, step):
    """Writes x [T, Hkv, d] into the numpy 4-bit pool at slots (those in range)."""
    nb, hkv, groups, _, w = pool.shape
    d, bs = w // 9, groups * 16
    code, scale = quantise(x, step)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    for t, slot in enumerate(slots):
        if not 0 <= slot < nb * bs:
            continue
        b, g, r = slot // bs, slot % bs // 16, slot % 16
        pool[b, :, g, which, r * (d // 2):(r + 1) * (d // 2)] = packed[t]
        at = 8 * d + r * (d // 16)
        pool[b, :, g, which, at:at + d // 16] = scale[t]


def decode(q, pool, table, seqs, scale):
    """step_reference.window_attention of one query per request over a fp64 pool."""
    return ref.window_attention(q.double(), pool, table, np.arange(len(seqs) + 1), seqs, scale, BIG,
                                0)


def weight_sums(q, pool, table, seqs, scale, refs, before):
    """(sums, allowance) [N, Hkv, cap] in fp64 after one step."""
    n, hq, d = q.shape
    bs, hkv = pool.shape[2], pool.shape[3]
    grp = hq // hkv
    _, lse, _, _, X, _ = refs
    out, tol = before.double().clone(), torch.zeros_like(before, dtype=torch.float64)
    for i in range(n):
        m = int(seqs[i])
        if m == 0:
            continue
        key = torch.arange(m, device=q.device)
        blk = torch.as_tensor(np.asarray(table[i]), device=q.device).long()[key // bs]
        for h in range(hkv):
            hs = slice(h * grp, (h + 1) * grp)
            x = q[i, hs].double() @ pool[blk, 0, key % bs, h].T * scale
            w = torch.exp(x - lse[i, hs, None])
            logit = (d + 8) * 2.0 ** -24 * X[i, hs, None]
            off = 2 * logit + 2.0 ** -20 * (1 + x.abs() + lse[i, hs, None].abs())
            out[i, h, :m] += w.sum(0)
            tol[i, h, :m] = (w * torch.expm1(off)).sum(0) + (grp + 1) * 2.0 ** -24 * out[i, h, :m] \
                + 1e-37
    return out, tol


def evict(scores, seqs, table, bs, budget, recent, first):
    """(kept [N][Hkv] lists, new lengths, freed block ids) of numpy arguments."""
    n, hkv, _ = scores.shape
    kept, lens, back = [], [], []
    for i in range(n):
        m = int(seqs[i])
        keep = min(m, budget)
        lens.append(keep)
        back += [int(b) for b in table[i, -(-keep // bs):-(-m // bs)]]
        kept.append([])
        for h in range(hkv):
            if m <= budget:
                kept[i].append(list(range(m)))
                continue
            mid = list(range(first, m - recent))
            s = scores[i, h]
            mid.sort(key=lambda p: (math.inf if math.isnan(s[p]) else -s[p], p)
                     if not math.isnan(s[p]) else (math.inf, p))
            # (NaN below everything, -inf included.)
            real = [p for p in mid if not math.isnan(s[p])]
            mid = (real + [p for p in mid if math.isnan(s[p])])[:budget - first - recent]
            kept[i].append(sorted(list(range(first)) + mid + list(range(m - recent, m))))
    return kept, lens, back


def prompts(q, k, v, qsl, scale):
    """window_attention of packed prompts (each a block of its own)."""
    lens = np.diff(qsl)
    bs = max(1, int(lens.max(initial=1)))
    hkv, d = k.shape[1:]
    pool = torch.zeros((len(lens), 2, bs, hkv, d), dtype=torch.float64, device=q.device)
    for i, m in enumerate(lens):
        pool[i, 0, :m] = k[qsl[i]:qsl[i] + m].double()
        pool[i, 1, :m] = v[qsl[i]:qsl[i] + m].double()
    return ref.window_attention(q.double(), pool, np.arange(len(lens))[:, None], qsl, lens, scale,
                                BIG, 0)
