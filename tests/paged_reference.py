"""The paged cache in 64 bits: a pool filled through the library, read back
with numpy, and attention over it from the definition, with the tolerance that
the kernels' stated roundings allow.

Tolerance of attention (before any run; u the output type's half step, 2^-11 the
fp16 half step).  The kernels round q~ and k_hat (code * scale) to fp16, p and
v_hat to fp16, and on the way out o and the rotation's entries to fp16, each
independently and by at most 2^-11 of the value, so by 2^-11 / sqrt 3 in the
root mean square:
  score t     sigma_s = 2^-11 sqrt(2/3) sm_scale sqrt(sum_i q~_i^2 k_ti^2), the largest over t taken for all;
  output i    e_i = sigma_s sum_t p_t |v_t - o|_i + 2^-11 sqrt(2/3) (sum_t p_t |v_t|_i + |o_i|);
the rotation back is orthogonal, so an output coordinate's error has the root
mean square |e|_2 / sqrt d; eight of those are allowed, plus the output's own
rounding u |x|, the fp16 subnormals of p (2^-25 a token against a sum of at
least 1) and fp32 arithmetic (2^-18 of the row)."""

from __future__ import annotations

import numpy as np
import torch

from oracle import srft_oracle as O

HALF_STEP = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
H16 = 2.0**-11


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def garbage(pages, seed):
    """Random codes, and scales that are NaN (e8m0: 255, an infinity): what unwritten rows may hold."""
    g = torch.Generator(device=pages.codes.device)
    g.manual_seed(seed)
    pages.codes.random_(0, 256, generator=g)
    if pages.scale_format == "e8m0":
        pages.scales.fill_(255)
    else:
        pages.scales.fill_(float("nan"))


def scales64(pages) -> np.ndarray:
    raw = pages.scales.cpu().numpy()
    return O.decode_scales(raw.view(np.uint16) if pages.scale_format == "fp16" else raw, pages.scale_format) \
        if pages.scale_format != "fp32" else raw.astype(np.float64)


def held_rows(pages, slots) -> np.ndarray:
    """z values [n][H][d] of the rows in `slots` (a list of ints), from the pool's bytes."""
    page = pages.codes.shape[2]
    s = np.asarray(slots)
    codes = pages.codes.cpu().numpy()[s // page, :, s % page]
    sc = scales64(pages)[s // page, :, s % page]
    return O.unpack_codes(codes, pages.bits).astype(np.float64) * np.repeat(sc, pages.group, axis=-1)


def lam64(pages) -> np.ndarray:
    return np.ones((pages.codes.shape[1], pages.d)) if pages.lam is None else f64(pages.lam)


def dequant_tolerance(z, lam, x, dtype):
    """z / lambda and R rounded to fp16 (2^-11 each of a unit-norm column), the output to its type."""
    norm = np.linalg.norm(z / lam, axis=-1, keepdims=True)
    return HALF_STEP[dtype] * np.abs(x) * 1.001 + 2.0**-10 * norm + 1e-6 * norm


def attention64(q, kp, vp, table, lens, qlens, seed, dtype, window=0, sm_scale=None):
    """(out, tol) [sum qlens][Hq][d] in 64 bits."""
    q = f64(q)
    Hq, d = q.shape[1:]
    H, page = kp.codes.shape[1:3]
    rep = Hq // H
    sm = 1 / np.sqrt(d) if sm_scale is None else sm_scale
    qt = O.rotate(q, seed, kp.transform)
    lk, lv = lam64(kp), lam64(vp)
    out, tol = np.zeros_like(q), np.zeros_like(q)
    first = 0
    for b, (n, m) in enumerate(zip(lens, qlens)):
        t = np.arange(n)
        slots = table[b, t // page].astype(np.int64) * page + t % page if n else np.zeros(0, np.int64)
        K = held_rows(kp, slots) if n else None
        V = held_rows(vp, slots) if n else None
        for i in range(m):
            pos = n - m + i
            lo = max(0, pos - window + 1) if window else 0
            if pos < lo or pos < 0:
                continue
            for h in range(Hq):
                g = h // rep
                k, v = K[lo:pos + 1, g], V[lo:pos + 1, g]
                qh = qt[first + i, h] / lk[g]
                s = sm * (k @ qh)
                p = np.exp(s - s.max())
                p /= p.sum()
                o = p @ v
                sig = H16 * np.sqrt(2 / 3) * sm * np.sqrt((k * k) @ (qh * qh)).max()
                e = sig * (p @ np.abs(v - o)) + H16 * np.sqrt(2 / 3) * (p @ np.abs(v) + np.abs(o))
                e = (e + len(p) * 2.0**-25 * np.abs(v).max(0)) / lv[g]
                x = O.unrotate(o / lv[g], seed, vp.transform)
                out[first + i, h] = x
                tol[first + i, h] = (HALF_STEP[dtype] * np.abs(x) + 8 * np.linalg.norm(e) / np.sqrt(d)
                                     + 2.0**-18 * np.linalg.norm(x))
        first += m
    return out, tol


class Cache:
    """A pool of shuffled pages holding given lengths, written through the library."""

    def __init__(self, K, lens, H, d, bits_k, bits_v, group, fmt, page, dtype, seed=3, lam=False, transform="srft",
                 transform_v=None, data_seed=1, most=None, gain=4.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(data_seed)
        self.page, self.lens, self.seed, self.dtype = page, list(lens), seed, dtype
        per = [-(-n // page) for n in lens]
        n_pages = sum(per) + 2
        most = most or max(max(per), 1)
        order = torch.randperm(n_pages, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), most), -7, dtype=torch.int32, device="cuda")  # unused entries: not read
        at = 0
        for b, c in enumerate(per):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.sides, self.rows = [], []
        for i, bits in enumerate((bits_k, bits_v)):
            lt = torch.exp(0.5 * torch.randn(H, d, generator=g, device="cuda")) if lam else None
            tr = transform if i == 0 or transform_v is None else transform_v
            p = K.alloc_pages(n_pages, page, H, d, bits, group, transform=tr, scale_format=fmt, lam=lt)
            garbage(p, 5 + i)
            x = torch.randn(sum(lens), H, d, generator=g, device="cuda")
            x[:, :, torch.randint(0, d, (2,), generator=g, device="cuda")] *= gain
            self.sides.append(p)
            self.rows.append(x.to(dtype))
        self.slots = self.slots_of([(b, 0, n) for b, n in enumerate(lens)])
        K.srft_kv_quantize_paged(self.sides[0], self.rows[0], self.sides[1], self.rows[1], self.slots, seed)

    def slots_of(self, spans):
        """int64 slots of tokens [lo, hi) of sequences, in order."""
        out = []
        for b, lo, hi in spans:
            t = torch.arange(lo, hi, device="cuda")
            out.append(self.table[b, t // self.page].long() * self.page + t % self.page)
        return torch.cat(out) if out else torch.zeros(0, dtype=torch.int64, device="cuda")

    def batch(self, K, qlens=None, lens=None, **kw):
        lens = self.lens if lens is None else lens
        seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if qlens is None:
            return K.PagedBatch(self.table, seq, **kw)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(qlens)]), dtype=torch.int32, device="cuda")
        kw.setdefault("total_q", int(sum(qlens)))
        kw.setdefault("max_q", max(qlens))
        return K.PagedBatch(self.table, seq, cu, **kw)


def attend(K, cache, q, batch, window=0, sm_scale=0.0, out=None, seed=None):
    k, v = cache.sides
    out = torch.empty_like(q) if out is None else out
    ws = torch.empty(max(16, K.q4kv_paged_attention_workspace_size(k, q.shape[1], batch, window)), dtype=torch.uint8,
                     device="cuda")
    K.q4kv_paged_attention(q, out, k, v, batch, sm_scale, window, cache.seed if seed is None else seed, ws)
    return out


def check(out, ref, tol):
    got = f64(out)
    assert np.isfinite(got).all()
    worst = np.abs(got - ref) - tol
    at = np.unravel_index(np.argmax(worst), worst.shape)
    assert worst.max() <= 0, f"off by {abs(got - ref)[at]:.3g} at {at}, allowed {tol[at]:.3g} (value {ref[at]:.3g})"
