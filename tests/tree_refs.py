"""Plain 64-bit statements of the speculative step's operators: rotation, tree attention and the
acceptance of a drafted path. Shares no code with the library."""
import math

import torch

D, PAGE = 128, 64


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the least step below the normal numbers (bf16: flushed ones count whole)."""
    return torch.finfo(dtype).tiny if dtype == torch.bfloat16 else 2.0 ** -25


# ---- rotation -----------------------------------------------------------------------------------
def rotated64(x, places, inv_freq, interleaved=False, scale=1.0):
    """Rows x [T, heads, 128] turned by their places [T], and the bound of what the library may be off.

    The angle in turns: p f / 2 pi from a two-part product, off by 2^-26 from its last sum and less than
    2^-27 from the parts while p f < 2^21: 2^-25.4 turns or 2^-22.7 of arc. sincospi and the factor add
    2^-23 together: 2^-22 on a cosine or sine. Product and sum: 2^-23 of the magnitudes. So 2^-21 (|x| +
    |y|) before the one rounding to dtype."""
    y = x.double().clone()
    err = torch.zeros_like(y)
    if inv_freq is not None:
        f = inv_freq.double()
        n = f.numel()
        a = torch.arange(n) * 2 if interleaved else torch.arange(n)
        b = a + 1 if interleaved else a + n
        angle = places.double()[:, None] * f.to(places.device)
        c, s = angle.cos()[:, None] * scale, angle.sin()[:, None] * scale
        xa, xb = x.double()[..., a], x.double()[..., b]
        y[..., a], y[..., b] = xa * c - xb * s, xa * s + xb * c
        size = (xa.abs() + xb.abs()) * abs(scale) * 2.0 ** -21
        err[..., a], err[..., b] = size, size
        h = half_step(x.dtype)
        err[..., a] += h * y[..., a].abs() + h * size + tiny(x.dtype)
        err[..., b] += h * y[..., b].abs() + h * size + tiny(x.dtype)
    return y, err


# ---- trees --------------------------------------------------------------------------------------
def make_parents(kind, n, gen):
    """Parents of n nodes."""
    if n == 0:
        return []
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "star":
        return [-1] + [0] * (n - 1)
    if kind == "forest":
        return [-1 if i % 5 == 0 else int(torch.randint(max(0, i - 6), i, (1,), generator=gen))
                for i in range(n)]
    if kind == "binary":
        return [(i - 1) // 2 if i else -1 for i in range(n)]
    assert kind == "random"
    return [-1] + [int(torch.randint(max(0, i - 8), i, (1,), generator=gen)) for i in range(1, n)]


def related(parents):
    """bool [n, n]: u is i or an ancestor of i; and the depths."""
    n = len(parents)
    mine, depth = torch.zeros((n, n), dtype=torch.bool), []
    for i, p in enumerate(parents):
        if 0 <= p < i:
            mine[i] = mine[p]
            depth.append(depth[p] + 1)
        else:
            depth.append(0)
        mine[i, i] = True
    return mine, torch.tensor(depth, dtype=torch.long)


def attention64(q, k, v, seq_lens, cu_q, block_table, parents, *, window=0, keep=None, sm=None,
                max_blocks=None):
    """out f64 [T, Hq, 128], lse f64 [T, Hq], and what rounding errors scale with: A = max_j sm sum_c |q_c
    K_jc|, W = sum_j p_j |V_j| and U = sum_j |V_j| over the visible tokens. Rows that belong to nobody are
    nan. parents: a list over all rows, or None."""
    T, Hq, _ = q.shape
    P, Hkv = k.shape[:2]
    G = Hq // Hkv
    sm = 1 / math.sqrt(D) if sm is None else sm
    dev = q.device
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=dev)
    wabs, usum = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=dev)
    amax = torch.zeros_like(lse)
    for b, n in enumerate(seq_lens):
        t0, t1 = cu_q[b], cu_q[b + 1]
        nq = t1 - t0
        if nq <= 0:
            continue
        n = min(n, block_table.shape[1] * PAGE)
        if n < nq:
            out[t0:t1], lse[t0:t1] = 0.0, -math.inf
            continue
        first = n - nq
        mine, depth = related([i - 1 for i in range(nq)] if parents is None else parents[t0:t1])
        see = torch.ones((nq, n), dtype=torch.bool)
        see[:, first:] = mine
        place = torch.arange(n)
        place[first:] = first + depth
        if window:
            see &= place[None] > place[first:, None] - window
        nb = (n + PAGE - 1) // PAGE
        bt = block_table[b, :nb].long().cpu()
        fine = (bt >= 0) & (bt < P)
        see &= fine.repeat_interleave(PAGE)[:n][None]
        pages = torch.where(fine, bt, torch.zeros_like(bt)).to(dev)
        for h in range(Hkv):
            mask = see.to(dev)
            if keep is not None:
                mask = mask & (keep[b, h, :nb].to(dev) != 0).repeat_interleave(PAGE)[:n][None]
            seen = mask.any(0)[:, None]
            K = torch.where(seen, k[pages, h].double().reshape(-1, D)[:n], 0.0)
            V = torch.where(seen, v[pages, h].double().reshape(-1, D)[:n], 0.0)
            for g in range(G):
                qq = q[t0:t1, h * G + g].double()
                s = (sm * (qq @ K.T)).masked_fill(~mask, -math.inf)
                a = (sm * (qq.abs() @ K.abs().T)).masked_fill(~mask, 0.0)
                z = torch.logsumexp(s, -1)
                base = torch.where(z == -math.inf, torch.zeros_like(z), z)
                p = torch.where(mask, torch.exp(s - base[:, None]), 0.0)
                clean = torch.nan_to_num(V, nan=0.0, posinf=0.0, neginf=0.0)
                out[t0:t1, h * G + g] = p @ clean
                wabs[t0:t1, h * G + g] = p @ clean.abs()
                usum[t0:t1, h * G + g] = mask.double() @ clean.abs()
                lse[t0:t1, h * G + g] = z
                amax[t0:t1, h * G + g] = a.max(-1).values
    return out, lse, amax, wabs, usum


def tolerance(out, lse, amax, wabs, usum, dtype):
    """Bounds of |library - 64 bits| for the output and the log-sum-exp.

    Scores: exact products of 16-bit numbers and 128 fp32 additions, each off by at most 2^-23 of the sum
    of magnitudes (the matrix unit truncates): ds = 2^-16 A, and the factor to log2 units and the difference
    to the reference another 2^-22 of the score, within it. Probabilities: e^ds - 1 (numerator and
    denominator: twice), one rounding to dtype, and the exponential's own 2^-20. In fp16 the largest enters
    as at least 2^7, so one below 2^-14 is rounded by half of the least step, 2^-25: 2^-32 U. bf16 has
    fp32's range: 2^-100 U. Output: one rounding. The sum is over positives in fp32: 2^-18 covers its additions,
    the joining of parts and the logarithm."""
    ds = amax * 2.0 ** -16
    half = half_step(dtype)
    rel = (half + 2.0 ** -18 + 2.2 * ds)[..., None]
    least = 2.0 ** -32 if dtype == torch.float16 else 2.0 ** -100
    return (half * out.abs() + (rel * wabs + least * usum) * (1 + half) + tiny(dtype),
            ds * 1.1 + 2.0 ** -18 + 2.0 ** -22 * lse.abs())


# ---- acceptance ---------------------------------------------------------------------------------
def accepted_path(draft, target, parents):
    """Nodes of the deepest path that the targets confirm (lists of one sequence)."""
    best = []
    for i in range(len(draft)):
        chain, u = [i], i
        while 0 <= parents[u] < u:
            u = parents[u]
            chain.append(u)
        chain.reverse()
        if chain[0] == 0 and all(draft[y] == target[x] for x, y in zip(chain, chain[1:])):
            if len(chain) > len(best):
                best = chain
    return best
