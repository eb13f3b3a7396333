"""Timed cases of the paged packed cache: writing K and V rows into pages, reading them back, and attention of
one or many query tokens a sequence over the pages.

A pool of pages holds one side (K or V) of the cache of all sequences of one layer: ``codes`` uint8
[n_pages][H][page_size][d*bits/8] and ``scales`` [n_pages][H][page_size][d/group], rows encoded as
z = lambda * R diag(s) x, one absmax scale a group, signed 4- or 8-bit codes.  A slot is page * page_size +
offset; a sequence's block table lists its pages in order.

Kinds of a case (one pass each):
  step    a decode step: the new token of every sequence is written into its slot, then attention over the pages
  attend  attention alone: one token a sequence, a few (verifying a draft), a chunk, or a whole prompt (causal)
  round   a prompt's rows are written into their slots and read back
  read    cached rows are read back
With ``own`` false ``run`` computes all of it from elementary torch operations in 32 bits, with ``own`` true it
calls the library.
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
SCALES = {"fp32": torch.float32, "fp16": torch.float16, "e8m0": torch.uint8}


def _case(name, kind, B, qlen, lo, hi, Hq, Hkv, d, bk, bv, group, scales, dtype, page, window=0, lam=False,
          srht=False):
    c = dict(kind=kind, B=B, qlen=qlen, lo=lo, hi=hi, Hq=Hq, Hkv=Hkv, d=d, bits_k=bk, bits_v=bv, group=group,
             scales=scales, dtype=dtype, page=page, window=window, lam=lam, srht=srht)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's chat on the small two-kv-head shape: latency of a step
        _case("step_one_chat", "step", 1, 1, 701, 701, 12, 2, 128, 4, 4, 16, "fp16", "fp16", 16, lam=True),
        # a serving batch of ragged lengths, 8-bit keys with 4-bit values
        _case("step_batch_k8v4", "step", 24, 1, 1, 9215, 32, 8, 128, 8, 4, 16, "fp32", "bf16", 16),
        # long contexts, one token each: the bytes of the cache
        _case("decode_long_b16", "attend", 16, 1, 131072, 131072, 32, 8, 128, 4, 4, 16, "fp16", "bf16", 64),
        # d = 256, one kv head, a sliding window layer
        _case("decode_d256_window", "attend", 8, 1, 600, 4096, 4, 1, 256, 4, 4, 32, "e8m0", "bf16", 32, window=512),
        # five drafted tokens a sequence verified at once
        _case("verify_5_tokens", "attend", 8, 5, 9000, 32768, 32, 8, 128, 4, 4, 16, "fp16", "bf16", 32),
        # the last chunk of a long prompt, per-channel lambda
        _case("chunk_2k_at_32k", "attend", 1, 2048, 32768, 32768, 12, 2, 128, 4, 4, 16, "fp32", "bf16", 64, lam=True),
        # a batch of whole prompts of odd lengths
        _case("prompts_ragged", "attend", 5, 0, 1, 4219, 32, 8, 128, 8, 4, 16, "fp16", "bf16", 16),
        # one long prompt at d = 64 with 8-bit codes and the Hadamard rotation
        _case("prompt_8k_d64_k8v8", "attend", 1, 0, 8191, 8191, 16, 4, 64, 8, 8, 16, "fp16", "bf16", 128, srht=True),
        # a short prompt cached and read back: latency of the two codec calls
        _case("round_short_d64", "round", 1, 0, 33, 33, 4, 2, 64, 8, 8, 32, "fp32", "fp16", 16),
        # a prompt of the d = 256 shape
        _case("round_d256", "round", 1, 0, 1537, 1537, 4, 1, 256, 4, 4, 16, "e8m0", "fp16", 64, lam=True),
        # a batch of prompts
        _case("round_prompts_8k", "round", 4, 0, 1000, 2911, 32, 8, 128, 8, 4, 16, "fp16", "bf16", 16),
        # a long cached context read back for a layer that wants plain rows
        _case("read_128k", "read", 1, 0, 131072, 131072, 32, 8, 128, 4, 4, 16, "fp16", "bf16", 64),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["step", "attend", "attend", "attend", "round", "read"])
    d = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 3, 4, 6, 7, 8])
    if kind in ("round", "read"):
        B, qlen, hi = log(1, 8), 0, log(16, 16384)
    else:
        mode = rng.choice(["one", "few", "chunk", "prompt"]) if kind == "attend" else "one"
        B = {"one": log(1, 64), "few": log(1, 16), "chunk": log(1, 3), "prompt": log(1, 5)}[mode]
        hi = {"one": log(16, 40000), "few": log(64, 20000), "chunk": log(1500, 20000), "prompt": log(64, 4000)}[mode]
        qlen = {"one": 1, "few": log(2, 16), "chunk": log(17, 1200), "prompt": 0}[mode]
    lo = max(1, int(hi * rng.choice([0.1, 0.5, 1.0])))
    group = rng.choice([16, 16, 32, d])
    window = rng.choice([0, 0, 0, log(16, 4096)]) if kind in ("step", "attend") else 0
    case = _case(None, kind, B, qlen, lo, hi, Hq, Hkv, d, rng.choice([4, 8]), rng.choice([4, 4, 8]), group,
                 rng.choice(["fp32", "fp16", "e8m0"]), rng.choice(["fp16", "bf16", "bf16", "bf16"]), rng.choice([16, 32, 64, 128]),
                 window=window, lam=rng.random() < 0.3, srht=rng.random() < 0.2)
    while work(case)["bytes"] > 1.5e9 or work(case)["flops"] > 3.5e11:  # no more than the largest listed cases
        case["hi"], case["lo"] = case["hi"] * 2 // 3, max(1, case["lo"] * 2 // 3)
        case["qlen"] = min(case["qlen"], case["hi"])
    return case


def _lengths(case):
    """Cached lengths and query lengths, from the case alone (the host knows them before a call)."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [lo + (hi - lo) * ((7 * b + 3) % max(B, 2)) // max(B - 1, 1) for b in range(B)]
    lens = [min(max(n, 1), hi) for n in lens]
    lens[-1] = hi
    q = [n if case["qlen"] == 0 else min(case["qlen"], n) for n in lens]
    return lens, q


# ---- the encoding, plain ----
def _signs(seed, d):
    """s_i = -1 where the top bit of output i of splitmix64(seed) is set."""
    mask, out = (1 << 64) - 1, []
    for i in range(d):
        z = (seed + (i + 1) * 0x9E3779B97F4A7C15) & mask
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & mask
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & mask
        out.append(-1.0 if (z ^ (z >> 31)) >> 63 else 1.0)
    return out


def _rotation(seed, d, srht):
    """The d x d matrix of the rotation, p = M x, in fp32 (entries formed in 64 bits)."""
    i = torch.arange(d, dtype=torch.int64)
    if srht:
        bits = (i[:, None] & i[None, :])
        par = sum((bits >> k) & 1 for k in range(d.bit_length())) & 1
        m = (1.0 - 2.0 * par.double()) / math.sqrt(d)
    else:
        ang = 2 * math.pi * ((i[: d // 2, None] * i[None, :]) % d).double() / d
        m = torch.empty(d, d, dtype=torch.float64)
        m[0::2] = math.sqrt(2 / d) * torch.cos(ang)
        m[1::2] = -math.sqrt(2 / d) * torch.sin(ang)
        m[0] = 1 / math.sqrt(d)
        m[1] = (1.0 - 2.0 * (i % 2).double()) / math.sqrt(d)
    return (m * torch.tensor(_signs(seed, d), dtype=torch.float64)[None, :]).float()


def _encode(x, rot, lam, bits, group, fmt):
    """Rows [n][H][d] -> packed codes [n][H][d*bits/8] and stored scales [n][H][d/group]."""
    n, H, d = x.shape
    q = 2 ** (bits - 1) - 1
    z = (x.float() @ rot.t()) * lam
    z = z.view(n, H, d // group, group)
    s = z.abs().amax(-1) / q
    if fmt == "fp32":
        stored = value = s
    elif fmt == "fp16":
        stored = s.clamp(max=65504.0).half()
        value = stored.float()
    else:
        m, e = torch.frexp(s)
        e = torch.where(m == 0.5, e - 1, e).clamp(-126, 127)
        stored = torch.where(s > 0, e + 127, torch.zeros_like(e)).to(torch.uint8)
        value = torch.where(s > 0, torch.ldexp(torch.ones_like(s), e), torch.zeros_like(s))
    c = torch.round(z / torch.where(value > 0, value, torch.ones_like(value))[..., None]).clamp(-q, q)
    c = torch.where(value[..., None] > 0, c, torch.zeros_like(c)).view(n, H, d).to(torch.int8)
    if bits == 4:
        c = (c[..., 0::2] & 15) | (c[..., 1::2] << 4)
    return c.view(torch.uint8), stored


def _values(codes, scales, bits, group, fmt):
    """Packed codes and stored scales -> the values z they stand for, fp32 [...][d]."""
    if bits == 4:
        c = codes.view(torch.int8)
        c = torch.stack(((c << 4) >> 4, c >> 4), -1).flatten(-2)
    else:
        c = codes.view(torch.int8)
    if fmt == "e8m0":
        s = torch.where(scales > 0, torch.ldexp(torch.ones((), device=scales.device), scales.int() - 127),
                        torch.zeros((), device=scales.device))
    else:
        s = scales.float()
    return (c.unflatten(-1, (-1, group)).float() * s[..., None]).flatten(-2)


def _write(st, side):
    p, slots, page = st[side], st["slots"], st["page"]
    codes, scales = _encode(p["x"], p["rot"], p["lam"], p["bits"], st["group"], st["scales"])
    p["codes"][slots // page, :, slots % page] = codes
    p["scales"][slots // page, :, slots % page] = scales


def _read(st, side):
    p, slots, page = st[side], st["slots"], st["page"]
    z = _values(p["codes"][slots // page, :, slots % page], p["scales"][slots // page, :, slots % page], p["bits"],
                st["group"], st["scales"])
    return ((z / p["lam"]) @ p["rot"]).to(st["dtype"])


def _attend(st):
    """Softmax attention over the pages, in the rotated coordinates (the rotation is orthogonal)."""
    k, v, page, d, q = st["k"], st["v"], st["page"], st["d"], st["q"]
    Hkv, rep = st["Hkv"], st["Hq"] // st["Hkv"]
    T = -(-max(st["lens"]) // page) * page
    table = st["table"][:, : T // page].long()
    B = table.shape[0]

    def rows(p):
        z = _values(p["codes"][table], p["scales"][table], p["bits"], st["group"], st["scales"])
        return z.transpose(1, 2).reshape(B, Hkv, T, d)  # [B][P][H][page][d] -> [B][H][P*page][d]

    M = st["max_q"]
    first, count = st["cu_q"][:-1].long(), (st["cu_q"][1:] - st["cu_q"][:-1]).long()
    i = torch.arange(M, device=q.device)
    at = (first[:, None] + i).clamp(max=q.shape[0] - 1)                      # [B][M] rows of q
    qr = (q.float() @ k["rot"].t())[at].view(B, M, Hkv, rep, d) / k["lam"][:, None]
    qr = qr.permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * rep, d) / math.sqrt(d)
    s = (qr @ rows(k).transpose(2, 3)).view(B, Hkv, M, rep, T)
    pos = (st["seq_lens"].long() - count)[:, None] + i                       # [B][M] positions of the query tokens
    t = torch.arange(T, device=q.device)
    seen = (t <= pos[..., None]) & (t < st["seq_lens"][:, None, None])
    if st["window"]:
        seen &= t > pos[..., None] - st["window"]
    s.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    den = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, M * rep, T) @ rows(v)).view(B, Hkv, M, rep, d) / torch.where(den > 0, den, 1)
    o = (o / v["lam"][:, None, None]) @ v["rot"]
    o = o.permute(0, 2, 1, 3, 4).reshape(B, M, Hkv * rep, d)
    return o[i < count[:, None]].to(st["dtype"])                             # rows of all sequences in order


# ---- states ----
def _rows(g, n, H, d, heavy):
    """K or V rows as a model makes them: unit normal, a few channels a head much larger."""
    x = torch.randn(n, H, d, generator=g, device="cuda")
    gain = torch.ones(H, d, device="cuda")
    ch = torch.rand(H, d, generator=g, device="cuda").topk(3, dim=1).indices
    gain.scatter_(1, ch, heavy)
    return x * gain


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    B, Hq, Hkv, d, page, group = (case[x] for x in ("B", "Hq", "Hkv", "d", "page", "group"))
    lens, ql = _lengths(case)
    dtype, fmt, kind = DTYPES[case["dtype"]], case["scales"], case["kind"]
    per = [-(-n // page) for n in lens]
    n_pages, most = sum(per) + 3, max(per)
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table, at = torch.zeros(B, most, dtype=torch.int32, device="cuda"), 0
    for b in range(B):
        table[b, : per[b]] = order[at : at + per[b]]
        at += per[b]
    seq = torch.tensor(lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + [sum(ql[: b + 1]) for b in range(B)], dtype=torch.int32, device="cuda")
    # the slots of the tokens of this pass: the query tokens, the last ones of each sequence (all, for round / read)
    pos = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, ql)])
    of = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(ql, device="cuda"))
    slots = table[of, pos // page].long() * page + pos % page
    n = int(sum(ql))
    st = dict(kind=kind, dtype=dtype, scales=fmt, page=page, group=group, d=d, Hq=Hq, Hkv=Hkv, lens=lens,
              max_q=max(ql), table=table, seq_lens=seq, cu_q=cu, slots=slots, window=case["window"],
              seed=17 + seed % 1000)
    rot = _rotation(st["seed"], d, case["srht"]).cuda()
    # the projection's output of this pass: q, k and v side by side a token
    qkv = torch.empty(n, (Hq + 2 * Hkv) * d, dtype=dtype, device="cuda")
    qkv[:, : Hq * d] = torch.randn(n, Hq * d, generator=g, device="cuda")
    st["q"] = qkv[:, : Hq * d].view(n, Hq, d)
    for i, name in enumerate("kv"):
        lam = torch.exp(0.5 * torch.randn(Hkv, d, generator=g, device="cuda")) if case["lam"] else None
        bits = case["bits_" + name]
        codes = torch.empty(n_pages, Hkv, page, d * bits // 8, dtype=torch.uint8, device="cuda")
        scales = torch.empty(n_pages, Hkv, page, d // group, dtype=SCALES[fmt], device="cuda")
        one = torch.ones(1, 1, device="cuda")
        for a in range(0, n_pages, max(1, (1 << 20) // (page * Hkv))):  # the cached rows, a million vectors at a time
            m = min(n_pages, a + max(1, (1 << 20) // (page * Hkv))) - a
            x = _rows(g, m * page, Hkv, d, 4.0)
            c, s = _encode(x, rot, one if lam is None else lam, bits, group, fmt)
            codes[a : a + m] = c.view(m, page, Hkv, -1).transpose(1, 2)
            scales[a : a + m] = s.view(m, page, Hkv, -1).transpose(1, 2)
        x = qkv[:, (Hq + i * Hkv) * d : (Hq + (i + 1) * Hkv) * d].view(n, Hkv, d)
        x.copy_(_rows(g, n, Hkv, d, 8.0))
        st[name] = dict(codes=codes, scales=scales, bits=bits, x=x, rot=rot, lam=one if lam is None else lam,
                        table_lam=lam, out=torch.empty(n, Hkv, d, dtype=dtype, device="cuda"))
    st["out"] = torch.empty(n, Hq, d, dtype=dtype, device="cuda")
    if own:  # the handles a user's program keeps: the pools, the batch's tables and the workspace
        import int8_kv_cache_srft_gb300 as K

        for name in "kv":
            p = st[name]
            p["pages"] = K.Pages(p["codes"], p["scales"], p["bits"], d=d, group=group, lam=p["table_lam"],
                                 transform="srht" if case["srht"] else "srft", scale_format=fmt)
        st["batch"] = K.PagedBatch(table, seq, cu, total_q=n, max_q=max(ql), max_seq_len=max(lens))
        need = K.q4kv_paged_attention_workspace_size(st["k"]["pages"], Hq, st["batch"], window=case["window"])
        st["work"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    return st


def run(st):
    kind, k, v = st["kind"], st["k"], st["v"]
    if own:
        import int8_kv_cache_srft_gb300 as K

        if kind in ("step", "round"):
            K.srft_kv_quantize_paged(k["pages"], k["x"], v["pages"], v["x"], st["slots"], st["seed"])
        if kind in ("round", "read"):
            K.srft_kv_dequantize_paged(k["pages"], k["out"], v["pages"], v["out"], st["slots"], st["seed"])
            return k["out"], v["out"]
        K.q4kv_paged_attention(st["q"], st["out"], k["pages"], v["pages"], st["batch"], 0.0, st["window"], st["seed"],
                               st["work"])
        return st["out"]
    if kind in ("step", "round"):
        _write(st, "k")
        _write(st, "v")
    if kind in ("round", "read"):
        return _read(st, "k"), _read(st, "v")
    return _attend(st)


def _pairs(case):
    """(query token, cached token) pairs that see each other, and the cached tokens that any query sees."""
    lens, ql = _lengths(case)
    w, pairs, seen = case["window"], 0, 0
    for n, m in zip(lens, ql):
        if w:
            lo = n - m  # positions lo .. n-1 see min(position + 1, w) tokens
            short = max(0, min(w, n) - lo)  # those that see all of the tokens before them
            pairs += short * lo + short * (short + 1) // 2 + (m - short) * w
            seen += min(n, m - 1 + w)
        else:
            pairs += m * (n - m) + m * (m + 1) // 2
            seen += n
    return pairs, seen


def work(case):
    lens, ql = _lengths(case)
    d, n = case["d"], sum(ql)
    row = sum(d * case["bits_" + s] // 8 + d // case["group"] * {"fp32": 4, "fp16": 2, "e8m0": 1}[case["scales"]]
              for s in "kv") * case["Hkv"]
    plain = 2 * 2 * d * case["Hkv"]  # 16-bit rows of K and V of one token
    kind = case["kind"]
    if kind == "round":  # each row is written, and read back with its codes
        return {"bytes": n * (2 * plain + 2 * row + 16), "flops": n * 4 * case["Hkv"] * 5 * d * math.log2(d)}
    if kind == "read":
        return {"bytes": n * (plain + row + 8), "flops": n * 2 * case["Hkv"] * 5 * d * math.log2(d)}
    pairs, seen = _pairs(case)
    table = sum(-(-m // case["page"]) for m in lens) * 4
    b = seen * row + n * case["Hq"] * d * 2 * 2 + table
    if kind == "step":
        b += n * (plain + row + 8)
    return {"bytes": b, "flops": 4 * d * case["Hq"] * pairs}


# ---- in 64 bits ----
def _turn64(x, seed, srht, back):
    """The rotation of rows x in 64 bits by transforms: an FFT of the signed row, or Hadamard butterflies."""
    d = x.shape[-1]
    s = torch.tensor(_signs(seed, d), dtype=torch.float64, device=x.device)
    if srht:
        y = x if back else x * s
        h = 1
        while h < d:
            y = y.reshape(*x.shape[:-1], d // (2 * h), 2, h)
            y = torch.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), -2)
            h *= 2
        y = y.reshape(x.shape) / math.sqrt(d)
        return y * s if back else y
    if back:
        f = torch.complex(x[..., 0::2], x[..., 1::2]) / math.sqrt(2)
        f = torch.cat((f, torch.zeros_like(f[..., :1])), -1)
        f[..., 0] = x[..., 0].to(f.dtype)
        f[..., -1] = x[..., 1].to(f.dtype)
        return torch.fft.irfft(f, n=d, norm="ortho") * s
    f = torch.fft.rfft(x * s, norm="ortho")
    p = torch.view_as_real(f[..., :-1]).flatten(-2) * math.sqrt(2)
    p[..., 0], p[..., 1] = f[..., 0].real, f[..., -1].real
    return p


def _levels64(z, bits, group, fmt):
    """The values that z is held as: nearest multiple of each group's stored scale, in 64 bits."""
    q = 2 ** (bits - 1) - 1
    zg = z.unflatten(-1, (-1, group))
    a = zg.abs().amax(-1, keepdim=True) / q
    if fmt == "fp32":
        a = a.float().double()
    elif fmt == "fp16":
        a = a.clamp(max=65504.0).half().double()
    else:
        a = torch.exp2(torch.ceil(torch.log2(a.clamp(min=2.0**-126)))) * (a > 0)
    return (torch.round(zg / a.clamp(min=1e-300)).clamp(-q, q) * a).flatten(-2)


def _held64(p, page_row, fmt, group):
    """One page row set's values in 64 bits, from its bytes."""
    raw = p["codes"][page_row].to(torch.int16)
    if p["bits"] == 4:
        lo, hi = raw % 16, raw // 16
        c = torch.stack((lo - 16 * (lo > 7), hi - 16 * (hi > 7)), -1).flatten(-2)
    else:
        c = raw - 256 * (raw > 127)
    s = p["scales"][page_row]
    s = torch.exp2(s.double() - 127) * (s > 0) if fmt == "e8m0" else s.double()
    return c.double() * s.repeat_interleave(group, -1)


def exact(case, seed):
    pairs, seen = _pairs(case)
    kind = case["kind"]
    if kind in ("step", "attend") and 4 * case["d"] * case["Hq"] * pairs > 4e12 or seen * case["Hkv"] > 3e7:
        return None  # the products would take minutes in 64 bits
    st = prepare(case, seed)
    srht, group, fmt, page, d = case["srht"], case["group"], case["scales"], case["page"], case["d"]
    new = {}
    for s in "kv":
        p = st[s]
        if kind in ("step", "round"):
            z = _levels64(_turn64(p["x"].double(), st["seed"], srht, False) * p["lam"].double(), p["bits"], group, fmt)
        else:
            slots = st["slots"]
            z = _held64(p, (slots // page, slice(None), slots % page), fmt, group)
        new[s] = z
    if kind in ("round", "read"):
        return tuple(_turn64(new[s] / st[s]["lam"].double(), st["seed"], srht, True) for s in "kv")
    rep, outs, first = case["Hq"] // case["Hkv"], [], 0
    q = _turn64(st["q"].double(), st["seed"], srht, False)
    lens, ql = _lengths(case)
    for b, (n, m) in enumerate(zip(lens, ql)):
        pages = st["table"][b, : -(-n // page)].long()
        held = {s: _held64(st[s], pages, fmt, group).transpose(0, 1).flatten(1, 2)[:, :n] for s in "kv"}
        if kind == "step":
            for s in "kv":
                held[s][:, n - m :] = new[s][first : first + m].transpose(0, 1)
        i, t = torch.arange(n - m, n, device="cuda")[:, None], torch.arange(n, device="cuda")
        hide = t > i
        if case["window"]:
            hide |= t <= i - case["window"]
        o = torch.empty(m, case["Hq"], d, dtype=torch.float64, device="cuda")
        for h in range(case["Hq"]):
            g = h // rep
            lk, lv = (st[s]["lam"][min(g, st[s]["lam"].shape[0] - 1)].double() for s in "kv")
            w = torch.softmax(((q[first : first + m, h] / lk) @ held["k"][g].t() / math.sqrt(d)).masked_fill(hide, -math.inf), -1)
            o[:, h] = w @ held["v"][g] / lv
        outs.append(_turn64(o, st["seed"], srht, True))
        first += m
    return torch.cat(outs)
