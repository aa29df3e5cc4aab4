"""Plain 64-bit statements of the 4-bit cache: the format, its records and attention over it.

Written from the format that include/ffd.h states, with explicit index tables; shares no code with
the library.
"""
import math

import torch

D, PAGE, GROUP, RECORD = 128, 64, 32, 5120


def quantise64(x):
    """codes int64 [..., 128], scale and off f64 [..., 4] of rows x [..., 128]."""
    g = x.double().reshape(x.shape[:-1] + (4, GROUP))
    lo, hi = g.min(-1).values, g.max(-1).values
    scale = ((hi - lo).float() / 15.0).half().double()
    off = (lo - 16 * scale).float().half().double()
    s, o = scale[..., None], off[..., None]
    t = torch.round((g - o) / torch.where(s > 0, s, torch.ones_like(s)))  # half to even
    c = torch.where(s > 0, t.clamp(16, 31) - 16, torch.zeros_like(t))
    return c.long().reshape(x.shape), scale, off


def values64(codes, scale, off):
    s = scale.repeat_interleave(GROUP, -1)
    o = off.repeat_interleave(GROUP, -1)
    return ((codes.double() + 16) * s + o).half().double()


def held64(x):
    """The values the cache holds for rows x."""
    return values64(*quantise64(x))


def byte_table():
    """Byte [64, 128] and nibble shift [128] of (token, channel), parameter byte [64, 4]."""
    byte = torch.zeros((PAGE, D), dtype=torch.long)
    shift = torch.zeros(D, dtype=torch.long)
    for c in range(D):
        J, within = divmod(c, 8)
        i, e = divmod(within, 2)
        nibble = i + 4 * e
        shift[c] = 4 * (nibble % 2)
        for r in range(PAGE):
            L = r // 2
            sector = (2 * (r % 2) + J // 8) ^ (L % 4)
            byte[r, c] = 128 * L + 32 * sector + 4 * (J % 8) + nibble // 2
    r = torch.arange(PAGE)[:, None]
    g = torch.arange(4)[None, :]
    return byte, shift, 4096 + 16 * r + 4 * g


BYTE, SHIFT, PARAM = byte_table()


def f16_bytes(x):
    """Low and high byte of the f16 value of x."""
    b = x.half().view(torch.int16).long() & 0xffff
    return b & 255, b >> 8


def put_rows(rec, page, row, head, x):
    """Write rows x [N, 128] of (page, row, head) [N] into records rec u8 [P, Hkv, 5120] (CPU)."""
    codes, scale, off = quantise64(x)
    for k in range(x.shape[0]):
        one = rec[page[k], head[k]]
        r = row[k]
        one[BYTE[r]] = 0
        for c in range(D):
            one[BYTE[r, c]] |= int(codes[k, c]) << int(SHIFT[c])
        for j, v in enumerate((scale[k], off[k])):
            lo, hi = f16_bytes(v)
            one[PARAM[r] + 2 * j] = lo.to(torch.uint8)
            one[PARAM[r] + 2 * j + 1] = hi.to(torch.uint8)


def pack64(x):
    """Records of whole pages x [P, Hkv, 64, 128], on x's device."""
    codes, scale, off = quantise64(x)
    rec = torch.zeros(x.shape[:2] + (RECORD,), dtype=torch.int64, device=x.device)
    byte, shift = BYTE.to(x.device), SHIFT.to(x.device)
    for c in range(D):
        rec[..., byte[:, c]] += codes[..., c] << shift[c]
    par = PARAM.to(x.device)
    for j, v in enumerate((scale, off)):
        lo, hi = f16_bytes(v)
        rec[..., par + 2 * j] = lo
        rec[..., par + 2 * j + 1] = hi
    return rec.to(torch.uint8)


def unpack64(rec):
    """Values f64 [..., 64, 128] that records hold."""
    r = rec.long()
    codes = (r[..., BYTE.to(rec.device)] >> SHIFT.to(rec.device)) & 15
    par = PARAM.to(rec.device)

    def f16(at):
        b = r[..., at] | (r[..., at + 1] << 8)
        return torch.where(b > 32767, b - 65536, b).to(torch.int16).view(torch.float16).double()
    return values64(codes, f16(par), f16(par + 2))


def attention64(q, k4, v4, seq_lens, cu_q, block_table, Hkv, *, window=0, keep=None, sm=None):
    """out f64 [T, Hq, 128], lse f64 [T, Hq], and per row and head the magnitudes that rounding
    errors scale with: A = max_j sm sum_c |q_c K_jc| and, per channel, W = sum_j p_j |V_j| and
    U = sum_j |V_j| over the tokens j that the row sees.
    Rows that belong to nobody are nan. Lists of python ints: seq_lens, cu_q."""
    T, Hq, _ = q.shape
    G = Hq // Hkv
    sm = 1 / math.sqrt(D) if sm is None else sm
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    wabs, usum = torch.zeros_like(out), torch.zeros_like(out)
    lse = torch.full((T, Hq), math.nan, dtype=torch.float64, device=q.device)
    amax = torch.zeros_like(lse)
    P = k4.shape[0]
    for b, n in enumerate(seq_lens):
        t0, t1 = cu_q[b], cu_q[b + 1]
        nq = t1 - t0
        if nq <= 0:
            continue
        nb = (n + PAGE - 1) // PAGE
        bt = block_table[b, :nb].long().cpu()
        fine = (bt >= 0) & (bt < P)
        pages = torch.where(fine, bt, torch.zeros_like(bt)).to(q.device)
        pos = torch.arange(n - nq, n, device=q.device)[:, None]
        j = torch.arange(n, device=q.device)[None]
        for h in range(Hkv):
            see = (j <= pos) & (pos >= 0)
            if window:
                see &= j > pos - window
            see &= fine.to(q.device).repeat_interleave(PAGE)[:n][None]
            if keep is not None:
                see &= (keep[b, h, :nb] != 0).repeat_interleave(PAGE)[:n][None]
            any_row = see.any(0)
            K = unpack64(k4[pages, h]).reshape(-1, D)[:n]
            V = unpack64(v4[pages, h]).reshape(-1, D)[:n]
            K = torch.where(any_row[:, None], K, torch.zeros_like(K))  # unused rows may be anything
            V = torch.where(any_row[:, None], V, torch.zeros_like(V))
            for g in range(G):
                qq = q[t0:t1, h * G + g].double()
                s = (sm * (qq @ K.T)).masked_fill(~see, -math.inf)
                a = (sm * (qq.abs() @ K.abs().T)).masked_fill(~see, 0.0)
                z = torch.logsumexp(s, -1)
                p = torch.where(see, torch.exp(s - torch.where(z == -math.inf, torch.zeros_like(z),
                                                               z)[:, None]), torch.zeros_like(s))
                out[t0:t1, h * G + g] = p @ V
                wabs[t0:t1, h * G + g] = p @ V.abs()
                usum[t0:t1, h * G + g] = see.double() @ V.abs()
                lse[t0:t1, h * G + g] = z
                amax[t0:t1, h * G + g] = a.max(-1).values if n else 0.0
    return out, lse, amax, wabs, usum


def tolerance(out, lse, amax, wabs, usum, dtype):
    """Bounds of |library - 64 bits| for the output and the log-sum-exp.

    Scores: products of f16 values and 128 fp32 additions, each off by at most 2^-23 of the sum of
    magnitudes (the matrix unit truncates): ds = 128 * 2^-23 A = 2^-16 A. Probabilities: e^ds - 1
    (numerator and denominator: twice), one rounding to f16 (half step 2^-11) and the exponential's
    own 2^-20. A probability enters as f16 of 2^7 at a reference that is at most the largest score, so
    that l >= 2^7 in the same unit; below 2^-14 it is rounded by half of f16's least step, 2^-25, or
    2^-32 of the row's largest: 2^-32 U. Output: one rounding to its type. The sum l is over positives
    in fp32: 2^-18 covers its additions and the logarithm."""
    ds = amax * 2.0 ** -16
    rel = (2.0 ** -11 + 2.0 ** -18 + 2.2 * ds)[..., None]
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny if dtype == torch.bfloat16 else 2.0 ** -25
    return (half * out.abs() + (rel * wabs + 2.0 ** -32 * usum) * (1 + half) + tiny,
            ds * 1.1 + 2.0 ** -18 + 2.0 ** -22 * lse.abs())
