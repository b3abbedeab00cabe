"""The 8-bit cache's operators from their definitions, in 64 bits and row by
row, sharing nothing with the kernels; and the error bounds of their outputs.

Bounds.  The kernels form scores from e4m3 bytes, which are exact in f16 and
bf16, and from queries in bf16 or in f16 with their row's largest magnitude
brought into [2^13, 2^14) by a power of two: bf16's 8 bits are exact there but
for f16's subnormals, half a step of 2^-25, so 2^-38 of the largest.  Sums are
float32.  Adding n products in any order, each addition off by at most one unit
of 2^-23 of the partial sum, is off by at most n 2^-23 sum|q k|; so a score is
off by

    ds <= scale (hd 2^-23 sum|q k| + 2^-38 max|q| sum|k|) + 2^-22 |s|

(the last term: the factors applied to it in float32).  A softmax weight is
then off by a factor exp(ds) and its rounding to f16 (2^-11; weights below
2^-22 of the row's largest by 2^-33 of it at most), its exponential by 2^-21.
The output adds half a bf16 step of its value, 2^-8."""

import math

import torch


def nearest8(y):
    """e4m3's nearest value, ties to even, saturating; float64 in and out."""
    _, e = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
    r = (torch.round(y / step) * step).clamp(-448.0, 448.0)
    return torch.where(torch.isinf(y), torch.copysign(torch.full_like(y, 448.0), y), r)


def scale_of(amax: float) -> float:
    e = -40
    while e < 40 and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def store(k8, scale, lens, x, block):
    """k8 [B, cap, g, hd] float64 values, scale [B, g, blocks]; rows x [B, n, g, hd]
    behind lens.  In place."""
    B, n, g, hd = x.shape
    for b in range(B):
        a = lens[b]
        for j in range(a // block, -(-(a + n) // block)):
            lo, first, end = j * block, max(j * block, a), min((j + 1) * block, a + n)
            for h in range(g):
                new = x[b, first - a:end - a, h]
                mag = new.abs()
                mag = mag[torch.isfinite(mag)]
                s = scale_of(float(mag.max()) if mag.numel() else 0.0)
                if first > lo:
                    old = float(scale[b, h, j])
                    s = max(s, old)
                    if s > old:
                        k8[b, lo:first, h] = nearest8(k8[b, lo:first, h] * (old / s))
                k8[b, first:end, h] = nearest8(new / s)
                scale[b, h, j] = s


def values(k8, scale, block):
    """[B, cap, g, hd] float64 of an e4m3 cache."""
    cap = k8.shape[1]
    return k8.double() * scale.double().repeat_interleave(block, 2)[:, :, :cap].transpose(1, 2)[..., None]


def visible(n_q, length, causal, device):
    end = torch.full((n_q,), length, device=device)
    if causal:
        end = length - n_q + 1 + torch.arange(n_q, device=device)
    return torch.arange(length, device=device) < end[:, None]


def attend(q, K, V, lens, causal, scale=None):
    """(o, lse, bound of o, bound of lse, ds) for q [B, n, H, hd] over the first
    lens[b] rows of K, V [B, cap, g, hd] (float64)."""
    q = q.double()
    B, n, H, hd = q.shape
    g = K.shape[2]
    scale = hd ** -0.5 if scale is None else scale
    o = torch.zeros((B, n, H, hd), dtype=torch.float64, device=q.device)
    lse = torch.full((B, H, n), -math.inf, dtype=torch.float64, device=q.device)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    ds_all = torch.zeros_like(lse)
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        see = visible(n, L, causal, q.device)
        for h in range(H):
            k, v = K[b, :L, h // (H // g)], V[b, :L, h // (H // g)]
            s = q[b, :, h] @ k.T * scale
            ds = scale * (hd * 2.0 ** -23 * (q[b, :, h].abs() @ k.abs().T)
                          + 2.0 ** -38 * q[b, :, h].abs().amax(-1, keepdim=True) * k.abs().sum(-1)) + 2.0 ** -22 * s.abs()
            s = s.masked_fill(~see, -math.inf)
            ds = (ds * see).amax(1)
            any_ = see.any(1)
            m = torch.where(any_, s.amax(1), 0.0)
            p = torch.exp(s - m[:, None])
            tot = p.sum(1)
            w = torch.where(any_[:, None], p / tot.clamp(min=1e-300)[:, None], 0.0)
            o[b, :, h] = w @ v
            lse[b, h] = torch.where(any_, m + torch.log(tot), -math.inf)
            A = w @ v.abs()
            top = w.amax(1, keepdim=True) * v.abs().sum(0)
            rel = (2.0 ** -11 + 2.0 ** -20 + 2.01 * ds)[:, None]
            bo[b, :, h] = 2.0 ** -8 * o[b, :, h].abs() + A * rel * 1.01 + 2.0 ** -33 * top
            bl[b, h] = ds * 1.01 + 2.0 ** -20 + 2.0 ** -22 * torch.where(any_, lse[b, h].abs(), 0.0)
            ds_all[b, h] = ds
    return o, lse, bo, bl, ds_all


def weigh(q, K, lse, lens, block, causal, weight, decay, scale=None):
    """(weight, bound) from the given lse."""
    q, lse = q.double(), lse.double()
    B, n, H, hd = q.shape
    g = K.shape[2]
    scale = hd ** -0.5 if scale is None else scale
    out, bound = weight.double().clone(), torch.zeros_like(weight, dtype=torch.float64)
    for b in range(B):
        L = int(lens[b])
        nb = -(-L // block)
        out[b, :, :nb] *= decay
        bound[b, :, :nb] = out[b, :, :nb].abs() * 2.0 ** -22
        if L == 0:
            continue
        see = visible(n, L, causal, q.device)
        which = torch.arange(L, device=q.device) // block
        for h in range(H):
            kv = h // (H // g)
            k = K[b, :L, kv]
            s = q[b, :, h] @ k.T * scale
            ds = scale * (hd * 2.0 ** -23 * (q[b, :, h].abs() @ k.abs().T)
                          + 2.0 ** -38 * q[b, :, h].abs().amax(-1, keepdim=True) * k.abs().sum(-1))
            ls = lse[b, h][:, None]
            live = see & torch.isfinite(ls)
            p = torch.where(live, torch.exp(s - torch.where(torch.isfinite(ls), ls, 0.0)), 0.0)
            out[b, kv].index_add_(0, which, p.sum(0))
            # factors and exponent in float32 (2^-22 of |s| and |lse|), the exponential, and the sums:
            # at most 16 + 32 additions deep for a thread's share of a tile, then n / 16 tiles
            err = p * (ds * 1.01 + 2.0 ** -21 * (s.abs() + ls.abs().clamp(max=1e30) + 1) + (64 + n) * 2.0 ** -24)
            bound[b, kv].index_add_(0, which, torch.where(live, err, 0.0).sum(0))
    return out, bound + 2.0 ** -23 * out.abs()


def evict(k8, v8, ks, vs, weight, lens, block, keep, first, last):
    """In place on k8, v8 (any dtype) and the scales; returns (weight, lens)."""
    B, cap, g, hd = k8.shape
    wout, lout = weight.clone(), list(lens)
    for b in range(B):
        L = lens[b]
        nb = -(-L // block)
        fixed = [j for j in range(nb) if j * block < first or (j + 1) * block > L - last or (j + 1) * block > L]
        for h in range(g):
            w = weight[b, h].tolist()
            free = [j for j in range(nb) if j not in set(fixed)]
            free.sort(key=lambda j: (-(math.inf if w[j] != w[j] else w[j]), w[j] == w[j], j))
            stay = sorted(fixed + free[:max(0, keep - len(fixed))])
            rows = [r for j in stay for r in range(j * block, min((j + 1) * block, L))]
            for t in (k8, v8):
                t[b, :len(rows), h] = t[b, rows, h].clone()
            for t in (ks, vs):
                t[b, h, :len(stay)] = t[b, h, stay].clone()
            wout[b, h, :len(stay)] = weight[b, h, stay]
            wout[b, h, len(stay):nb] = 0
            lout[b] = len(rows)
    return wout, lout
