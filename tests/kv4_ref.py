"""The 4-bit KV cache written out in plain 64-bit torch on the CPU, from the format and the
formulas in include/mixq.h: quantization of rows, the page bytes, reading rows back, and
attention with the error bound of the CUDA path beside it."""
from __future__ import annotations

import torch

PAIR_NAN = 0x7FFF


def page_bytes(page_size, D):
    return page_size * (D + 8)


def quantize(x):
    """Rows [..., D] of a 16-bit type -> (codes int64 [..., D], s, lo [..., 1] in that type).
    Codes are decided in fp32 (differences, 1/s and the product rounded once each)."""
    f = x.float()
    lo, hi = f.min(-1, keepdim=True).values, f.max(-1, keepdim=True).values
    rng = hi - lo
    s = (rng.double() / 15).float().to(x.dtype)  # 53 bits hold the fp32 quotient exactly enough
    s = torch.where(s.float() < 2.0 ** -126, torch.zeros_like(s), s)
    inv = torch.where(s > 0, s.float().reciprocal(), torch.zeros_like(lo))
    codes = torch.nan_to_num((f - lo) * inv).round().clamp(0, 15).long()
    bad = ~torch.isfinite(rng)
    nan = torch.full_like(s, float("nan"))
    return codes, torch.where(bad, nan, s), torch.where(bad, nan, lo.to(x.dtype))


def k_place(tok, dim, D):
    """(byte, shift) of a K code in its record."""
    nibble = dim % 8 // 2 + 4 * (dim % 2)
    return tok * (D // 2) + dim // 8 * 4 + nibble // 2, 4 * (nibble % 2)


def v_place(tok, dim, D):
    b = dim // 2
    i = 2 * (tok % 2) + tok // 8
    return 8 * D + b // 32 * 512 + b % 8 * 64 + tok % 8 // 2 * 16 + b // 8 % 4 * 4 + i, 4 * (dim % 2)


class Pages:
    """Page bytes on the CPU."""

    def __init__(self, pages, page_size, D, dtype):
        self.p, self.page_size, self.D, self.dtype = pages, page_size, D, dtype

    def _record(self, table_row, pos, head):
        page = int(table_row[pos // self.page_size])
        rec = 16 * (self.D + 8)
        at = pos % self.page_size // 16 * rec
        return self.p[page, head, at:at + rec], pos % 16

    def write(self, table_row, pos, k, v):
        """One token's rows [heads, D]."""
        D = self.D
        for h in range(k.shape[0]):
            rec, tok = self._record(table_row, pos, h)
            for x, place, at in ((k[h], k_place, 16 * D), (v[h], v_place, 16 * D + 64)):
                codes, s, lo = quantize(x)
                for d in range(D):
                    byte, shift = place(tok, d, D)
                    rec[byte] = (int(rec[byte]) & (0xF0 >> shift)) | int(codes[d]) << shift
                pair = torch.cat([s, lo]).view(torch.int16)
                if torch.isnan(s).any():
                    pair = torch.full((2,), PAIR_NAN, dtype=torch.int16)
                rec[at + 4 * tok:at + 4 * tok + 4] = pair.view(torch.uint8)

    def rows(self, table_row, positions, head):
        """fp64 K and V rows [n, D] of some positions."""
        D, P = self.D, self.page_size
        pos = torch.as_tensor(positions, dtype=torch.long)
        if len(pos) == 0:
            return torch.zeros((0, D), dtype=torch.float64), torch.zeros((0, D), dtype=torch.float64)
        raw = self.p[table_row[pos // P].long(), head]
        base = (pos % P // 16 * 16 * (D + 8))[:, None]
        tok, dim = (pos % 16)[:, None], torch.arange(D)[None]
        out = []
        for place, at in ((k_place, 16 * D), (v_place, 16 * D + 64)):
            byte, shift = place(tok, dim, D)
            code = raw.gather(1, base + byte).long() >> shift & 15
            pair = raw.gather(1, base + at + 4 * tok + torch.arange(4)[None]).flatten()
            pair = pair.view(self.dtype).view(-1, 2).double()
            out.append(code.double() * pair[:, :1] + pair[:, 1:])
        return out

    def scales(self, table_row, positions, head):
        pos = torch.as_tensor(positions, dtype=torch.long)
        raw = self.p[table_row[pos // self.page_size].long(), head]
        base = (pos % self.page_size // 16 * 16 * (self.D + 8))[:, None]
        res = []
        for at in (16 * self.D, 16 * self.D + 64):
            pair = raw.gather(1, base + at + 4 * (pos % 16)[:, None] + torch.arange(4)[None]).flatten()
            res.append(pair.view(self.dtype).view(-1, 2).double())
        return res


def visible(p, n, window, sinks):
    j = torch.arange(n)
    seen = j <= p
    if window > 0:
        seen &= (j > p - window) | (j < sinks)
    return seen


def attention(pages: Pages, q, table, lens, cu, scale, window=0, sinks=0):
    """fp64 outputs [rows, heads, D] and an elementwise bound on the CUDA path's error.

    The bound counts, for each output o = sum p (s c + lo) / sum p:
      half a step of the output type, eps/2 |o|;
      the rounding of weight times V's scale to fp16 before the product, 2^-11 of the code part
        A = sum p s c / sum p, and 2^-25 absolute for weights that fall below fp16's normal range
        (they are scaled so that the largest scale is at least 2^6): n 15 2^-25 2^-6 max s;
      errors of the scores: each is a sum of D products (fp32 accumulation, at most a step of
        2^-23 per term, of magnitudes up to sum |q| 15 s) and lo sum q, so a score is off by
        delta <= scale (D + 32) 2^-23 sum|q| (15 s + |lo|), which moves every weight by 2 delta
        relative, numerator and denominator together;
      the exponential (2^-22 relative, and 2^-23 of its argument's magnitude) and fp32 sums of n
        terms spread over lanes, warps and parts: 2^-17 (1 + n / 2048) of A + B covers both, with
        B = sum p |lo| / sum p;
      where a sequence has more than 32 rows per kv head, the tile kernel's operands: weights and V
        rows rounded once each to the type, so every term p v is off by at most 2 (eps/2) |p v|:
        eps C with C = sum p |v| / sum p (second-order terms are below the fp32 allowance above);
        for a bf16 cache the type of that product is fp16, or bf16 for records that do not fit it, whose
        weights are rounded to fp16 first: 2^-12 C more."""
    D = pages.D
    rows, heads = q.shape[0], q.shape[1]
    n_kv = pages.p.shape[1]
    group = heads // n_kv
    out = torch.zeros((rows, heads, D), dtype=torch.float64)
    tol = torch.zeros_like(out)
    eps = torch.finfo(pages.dtype).eps / 2
    for s in range(len(lens)):
        r0, r1 = (s, s + 1) if cu is None else (int(cu[s]), int(cu[s + 1]))
        n = int(lens[s])
        if r1 <= r0:
            continue
        for h in range(n_kv):
            k, v = pages.rows(table[s], range(n), h)
            if n:
                kp, vp = pages.scales(table[s], range(n), h)
            for i in range(r0, r1):
                p = n - (r1 - r0) + (i - r0)
                seen = visible(p, n, window, sinks)
                if not seen.any():
                    continue
                kk, vv, lo, sc = k[seen], v[seen], vp[seen, 1:], vp[seen, :1]
                qq = q[i, h * group:(h + 1) * group].double()
                z = qq @ kk.T * scale
                w = torch.softmax(z, -1)
                o = w @ vv
                out[i, h * group:(h + 1) * group] = o
                mag = (15 * kp[seen, 0].abs() + kp[seen, 1].abs()).max()
                delta = scale * (D + 32) * 2.0 ** -23 * qq.abs().sum(-1, keepdim=True) * mag
                delta = delta + 2.0 ** -23 * z.abs().amax(-1, keepdim=True)
                A = w @ (vv - lo)
                B = w @ lo.abs().expand_as(vv)
                m = int(seen.sum())
                tol[i, h * group:(h + 1) * group] = (
                    eps * o.abs() + 2.0 ** -11 * A.abs() + m * 15 * 2.0 ** -31 * sc.abs().max()
                    + (2 * delta + 2.0 ** -17 * (1 + m / 2048)) * (A.abs() + B)
                    + torch.finfo(pages.dtype).smallest_normal * eps)
                if (r1 - r0) * group > 32:
                    step = 2 * eps + (2.0 ** -12 if pages.dtype == torch.bfloat16 else 0.0)
                    tol[i, h * group:(h + 1) * group] += step * (w @ vv.abs())
    return out, tol


def assert_close(got, want, tol, what=""):
    got = got.double().cpu()
    same_nan = torch.isnan(got) == torch.isnan(want)
    assert bool(same_nan.all()), f"{what}: NaN in {int((~same_nan).sum())} wrong places"
    off = torch.nan_to_num((got - want).abs() - tol, nan=-1.0)
    if bool((off > 0).any()):
        at = int(off.argmax())
        raise AssertionError(f"{what}: {int((off > 0).sum())} of {off.numel()} outputs outside the bound; worst got "
                             f"{got.flatten()[at]} want {want.flatten()[at]} bound {tol.flatten()[at]}")

