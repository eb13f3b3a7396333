"""The paged cache against its definition in 64 bits: rows written into slots
and read back, and attention of ragged query rows over the pages."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import srft_oracle as O
from tests import paged_reference as R
from tests.parity import assert_codes

pytestmark = pytest.mark.gpu

K = None
HALF, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    global K
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import int8_kv_cache_srft_gb300 as mod

    mod.library()
    K = mod
    yield
    assert K.srftkv_device_fault() == 0


def rand(*shape, dtype, seed=1, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ---------------------------------------------------------------------------
# Writing and reading back
# ---------------------------------------------------------------------------
def near_boundary(a_over_q, fmt, tol=1e-5):
    a = np.asarray(a_over_q, dtype=np.float64)
    if fmt == "e8m0":
        p = np.ldexp(1.0, np.round(np.log2(np.where(a > 0, a, 1.0))).astype(np.int64))
        return (a > 0) & (np.abs(a - p) <= tol * a)
    h16 = np.clip(a, 0, O.FP16_MAX).astype(np.float16)
    h = h16.astype(np.float64)
    below = np.where(h <= a, h, np.nextafter(h16, np.float16(-np.inf)).astype(np.float64))
    above = np.where(h >= a, h, np.nextafter(h16, np.float16(np.inf)).astype(np.float64))
    return (a > 0) & (np.abs(a - (below + above) / 2) <= tol * a)


def check_written(pages, slots, x, seed):
    """Scales within 1e-5 (bit-exact away from a rounding boundary for fp16 and e8m0), codes of the stored scales."""
    lam = None if pages.lam is None else R.f64(pages.lam)
    enc = O.srft_kv_quantize(R.f64(x), lam, pages.bits, pages.group, seed, transform=pages.transform,
                             scale_format=pages.scale_format)
    s, page = slots.cpu().numpy(), pages.codes.shape[2]
    raw = pages.scales.cpu().numpy()[s // page, :, s % page]
    if pages.scale_format == "fp32":
        got = raw.astype(np.float64)
        assert np.all(np.abs(got - enc["scales"]) <= 1e-5 * enc["scales"] + 1e-30)
    else:
        raw = raw.view(np.uint16) if pages.scale_format == "fp16" else raw
        diff = raw != np.asarray(enc["scales_raw"])
        assert not (diff & ~near_boundary(enc["a_over_q"], pages.scale_format)).any()
        got = O.decode_scales(raw, pages.scale_format)
    got = np.repeat(got, pages.group, axis=-1)
    r = np.where(got > 0, enc["z"] / np.where(got > 0, got, 1.0), 0.0)
    assert_codes(pages.codes.cpu().numpy()[s // page, :, s % page], r, pages.bits)


CODEC = [  # d, bits_k, bits_v, group, fmt, page, dtype, lam, transform
    (64, 4, 4, 16, "fp32", 16, HALF, False, "srft"),
    (64, 8, 4, 64, "e8m0", 32, BF16, True, "srft"),
    (64, 8, 8, 32, "fp16", 16, BF16, False, "srht"),
    (128, 4, 4, 16, "fp16", 64, BF16, False, "srft"),
    (128, 8, 4, 16, "fp32", 16, HALF, True, "srft"),
    (128, 4, 8, 32, "e8m0", 16, HALF, False, "srht"),
    (128, 8, 8, 128, "fp16", 128, BF16, True, "srft"),
    (256, 4, 4, 16, "e8m0", 32, BF16, False, "srft"),
    (256, 8, 8, 64, "fp32", 16, HALF, True, "srht"),
    (256, 4, 8, 256, "fp16", 256, HALF, False, "srft"),
]


@pytest.mark.parametrize("n", [1, 7, 300])
@pytest.mark.parametrize("d,bk,bv,group,fmt,page,dtype,lam,tr", CODEC)
def test_write_and_read_back(d, bk, bv, group, fmt, page, dtype, lam, tr, n):
    H, n_pages, seed = 3, 2 * (-(-n // page)) + 3, 11
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    sides = [K.alloc_pages(n_pages, page, H, d, b, group, transform=tr, scale_format=fmt,
                           lam=torch.exp(0.5 * torch.randn(H, d, generator=g, device="cuda")) if lam else None)
             for b in (bk, bv)]
    for i, p in enumerate(sides):
        R.garbage(p, i)
    before = [(p.codes.clone(), p.scales.clone()) for p in sides]
    # K and V as slices of a fused projection; some tokens are padding
    fused = rand(n, (2 * H + 1) * d, dtype=dtype, seed=n + 1)
    fused[:, ::37] *= 20
    if n > 5:
        fused[4, d:(H + 1) * d] = 0  # a row of zeros: scale 0, codes 0
    xk = fused[:, d:(H + 1) * d].view(n, H, d)
    xv = fused[:, (H + 1) * d:].view(n, H, d)
    slots = torch.randperm(n_pages * page, generator=g, device="cuda")[:n]
    if n > 5:
        slots[2] = -1
    live = slots >= 0
    K.srft_kv_quantize_paged(sides[0], xk, sides[1], xv, slots, seed)
    for p, x in zip(sides, (xk, xv)):
        check_written(p, slots[live], x[live], seed)
    rest = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    rest[slots[live]] = False
    rest = rest.view(n_pages, page)
    for p, (c, s) in zip(sides, before):
        assert torch.equal(p.codes.transpose(1, 2)[rest], c.transpose(1, 2)[rest])
        assert torch.equal(p.scales.view(torch.uint8).transpose(1, 2)[rest], s.view(torch.uint8).transpose(1, 2)[rest])
    # back, into a strided buffer; rows of padding stay as they were
    back = torch.full((n, (2 * H + 1) * d), 3.0, dtype=dtype, device="cuda")
    yk, yv = back[:, d:(H + 1) * d].view(n, H, d), back[:, (H + 1) * d:].view(n, H, d)
    K.srft_kv_dequantize_paged(sides[0], yk, sides[1], yv, slots, seed)
    assert (back[:, :d] == 3).all() and (back[~live] == 3).all()
    for p, y in zip(sides, (yk, yv)):
        z, lm = R.held_rows(p, slots[live].cpu().numpy()), R.lam64(p)
        want = O.unrotate(z / lm, seed, p.transform)
        assert np.all(np.abs(R.f64(y[live]) - want) <= R.dequant_tolerance(z, lm, want, dtype))


@pytest.mark.parametrize("n", [2500, 20000])
@pytest.mark.parametrize("d,bk,bv,group,fmt,page,dtype,lam,tr", CODEC)
def test_large_calls(d, bk, bv, group, fmt, page, dtype, lam, tr, n):
    """Calls of thousands of tokens (other kernels than the small ones take): every row of the shorter call against the
    oracle and a fixed sample of the longer one, every row of both by what holds for any."""
    H, seed = 5, 21
    n_pages = -(-n // page) + 1
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    sides = [K.alloc_pages(n_pages, page, H, d, b, group, transform=tr, scale_format=fmt,
                           lam=torch.exp(0.5 * torch.randn(H, d, generator=g, device="cuda")) if lam else None)
             for b in (bk, bv)]
    for i, p in enumerate(sides):
        R.garbage(p, i)
    before = [p.codes.clone() for p in sides]
    fused = rand(n, 2 * H * d, dtype=dtype, seed=n + 1)
    fused[:, ::41] *= 12
    xk, xv = fused[:, :H * d].view(n, H, d), fused[:, H * d:].view(n, H, d)
    order = torch.randperm(n_pages, generator=g, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = order[t // page] * page + t % page  # runs of tokens in pages, as sequences write them
    slots[n // 3] = -1
    slots[n - 2] = -5
    K.srft_kv_quantize_paged(sides[0], xk, sides[1], xv, slots, seed)
    pick = torch.arange(n) if n <= 2500 else torch.cat(
        [torch.arange(0, 300), torch.randperm(n, generator=torch.Generator().manual_seed(1))[:2000],
         torch.arange(n - 300, n)]).unique()
    pick = pick.cuda()
    pick = pick[slots[pick] >= 0]
    for p, x in zip(sides, (xk, xv)):
        check_written(p, slots[pick], x[pick], seed)
    live = slots >= 0
    written = torch.zeros(n_pages * page, dtype=torch.bool, device="cuda")
    written[slots[live]] = True
    written = written.view(n_pages, page)
    for p, c in zip(sides, before):
        assert torch.equal(p.codes.transpose(1, 2)[~written], c.transpose(1, 2)[~written])
        sc = p.scales if fmt == "e8m0" else p.scales.float()
        sc = sc.transpose(1, 2)
        assert (sc[written] != 255).all() if fmt == "e8m0" else torch.isfinite(sc[written]).all()
    yk, yv = torch.full_like(fused, 3.0)[:, :H * d].view(n, H, d), torch.full((n, H, d), 3.0, dtype=dtype, device="cuda")
    K.srft_kv_dequantize_paged(sides[0], yk, sides[1], yv, slots, seed)
    for p, x, y in zip(sides, (xk, xv), (yk, yv)):
        assert (y[~live] == 3).all()
        z, lm = R.held_rows(p, slots[pick].cpu().numpy()), R.lam64(p)
        want = O.unrotate(z / lm, seed, p.transform)
        assert np.all(np.abs(R.f64(y[pick]) - want) <= R.dequant_tolerance(z, lm, want, dtype))
        # every row: |x_hat - x| <= |scale / (2 lambda)| (2-norms; scales below the e8m0 ceiling: twice the group's
        # largest step), with the roundings above
        step = (torch.exp2(p.scales.float() - 127) if fmt == "e8m0" else p.scales.float())
        step = step[slots[live] // page, :, slots[live] % page].repeat_interleave(group, -1) / 2
        if p.lam is not None:
            step = step / p.lam
        err = (y[live].float() - x[live].float()).norm(dim=-1)
        size = x[live].float().norm(dim=-1) + step.norm(dim=-1)
        half = R.HALF_STEP[dtype] + 2.0**-10 * d**0.5
        assert (err <= step.norm(dim=-1) + half * size + 1e-4).all()


def test_one_side_only_and_a_slot_read_twice():
    p = K.alloc_pages(4, 16, 2, 128, 4, 16)
    x = rand(5, 2, 128, dtype=BF16)
    slots = torch.tensor([3, 60, 17, 0, 31], device="cuda")
    K.srft_kv_quantize_paged(None, None, p, x, slots, 1)
    y = torch.empty(7, 2, 128, dtype=BF16, device="cuda")
    again = torch.tensor([3, 3, 60, 17, 0, 31, 31], device="cuda")
    K.srft_kv_dequantize_paged(p, y, None, None, again, 1)
    assert torch.equal(y[0], y[1]) and torch.equal(y[5], y[6])
    assert (y[torch.tensor([0, 2, 3, 4, 5])].float() - x.float()).abs().max() < 1


def test_slots_outside_the_pool_are_skipped_and_reported():
    p = K.alloc_pages(3, 16, 2, 128, 8, 16)
    R.garbage(p, 1)
    before = p.codes.clone()
    x = rand(4, 2, 128, dtype=HALF)
    slots = torch.tensor([48, 5, 1 << 40, -(1 << 40)], device="cuda")
    K.srft_kv_quantize_paged(p, x, None, None, slots, 1)
    assert K.srftkv_device_fault() == 1 << 16
    same = torch.ones(48, dtype=torch.bool, device="cuda")
    same[5] = False
    assert torch.equal(p.codes.transpose(1, 2)[same.view(3, 16)], before.transpose(1, 2)[same.view(3, 16)])
    y = torch.full((4, 2, 128), 2.0, dtype=HALF, device="cuda")
    K.srft_kv_dequantize_paged(p, y, None, None, slots, 1)
    assert K.srftkv_device_fault() == 1 << 16
    assert (y[[0, 2, 3]] == 2).all() and (y[1].float() - x[1].float()).abs().max() < 0.1


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
ATTN = [  # d, bits_k, bits_v, group, fmt, page, dtype, rep, lam, transform
    (64, 4, 4, 16, "fp32", 16, HALF, 1, False, "srft"),
    (64, 8, 8, 16, "fp16", 32, BF16, 4, True, "srht"),
    (64, 8, 4, 64, "e8m0", 16, BF16, 2, False, "srft"),
    (128, 4, 4, 16, "fp16", 16, BF16, 4, False, "srft"),
    (128, 4, 4, 16, "fp32", 64, HALF, 6, True, "srft"),
    (128, 8, 4, 16, "fp32", 32, BF16, 4, False, "srft"),
    (128, 4, 8, 32, "e8m0", 128, HALF, 3, False, "srht"),
    (128, 8, 8, 128, "fp16", 16, HALF, 8, True, "srft"),
    (256, 4, 4, 32, "e8m0", 32, BF16, 4, False, "srft"),
    (256, 8, 4, 16, "fp32", 16, HALF, 2, True, "srft"),
    (256, 4, 8, 256, "fp16", 64, BF16, 1, False, "srht"),
    (256, 8, 8, 16, "fp16", 16, BF16, 7, False, "srft"),
]


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("d,bk,bv,group,fmt,page,dtype,rep,lam,tr", ATTN)
def test_one_token(d, bk, bv, group, fmt, page, dtype, rep, lam, tr, window):
    H, lens = 2, [0, 1, 2, 15, 16, 17, 31, 33, 64, 129, 300]
    c = R.Cache(K, lens, H, d, bk, bv, group, fmt, page, dtype, lam=lam, transform=tr)
    q = rand(len(lens), H * rep, d, dtype=dtype, seed=4)
    out = R.attend(K, c, q, c.batch(K), window=window)
    ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), lens, [1] * len(lens), c.seed, dtype, window)
    assert (out[0] == 0).all()
    R.check(out, ref, tol)


@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("qlens", [[2, 1, 3, 5, 0, 4], [16, 9, 1, 13, 17, 8], [40, 64, 33, 0, 127, 65]])
@pytest.mark.parametrize("d,bk,bv,group,fmt,page,dtype,rep,lam,tr", ATTN)
def test_few_tokens(d, bk, bv, group, fmt, page, dtype, rep, lam, tr, qlens, window):
    """Query counts around the tile sizes, more query tokens than cached ones among them (the first see nothing)."""
    H, lens = 1, [130, 3, 200, 17, 64, 257]
    c = R.Cache(K, lens, H, d, bk, bv, group, fmt, page, dtype, lam=lam, transform=tr)
    q = rand(sum(qlens), H * rep, d, dtype=dtype, seed=4)
    out = R.attend(K, c, q, c.batch(K, qlens), window=window)
    ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), lens, qlens, c.seed, dtype, window)
    R.check(out, ref, tol)


@pytest.mark.parametrize("d,bk,bv,group,fmt,page,dtype,rep,lam,tr", ATTN)
def test_whole_prompts(d, bk, bv, group, fmt, page, dtype, rep, lam, tr):
    H, lens = 2, [1, 131, 260]
    c = R.Cache(K, lens, H, d, bk, bv, group, fmt, page, dtype, lam=lam, transform=tr)
    q = rand(sum(lens), H * rep, d, dtype=dtype, seed=4)
    out = R.attend(K, c, q, c.batch(K, lens))
    ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), lens, lens, c.seed, dtype)
    R.check(out, ref, tol)


@pytest.mark.parametrize("d,rep,m", [(128, 4, 1), (128, 16, 1), (128, 2, 30), (64, 5, 3), (256, 2, 4), (128, 1, 300)])
def test_long_contexts(d, rep, m):
    """Thousands of tokens (the work is split over them and joined), ragged, with a query's scale in play."""
    H, lens, qlens = 1, [5000, 2049, 7, 3333], [m, m, min(m, 7), 0]
    c = R.Cache(K, lens, H, d, 4, 4, 16, "fp16", 32, BF16)
    q = rand(sum(qlens), H * rep, d, dtype=BF16, seed=4, scale=2.0)
    out = R.attend(K, c, q, c.batch(K, qlens), sm_scale=0.11)
    pick = range(sum(qlens)) if m < 40 else None
    ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), lens, qlens, c.seed, BF16, 0, 0.11)
    assert pick is None or len(pick) == ref.shape[0]
    R.check(out, ref, tol)


@pytest.mark.parametrize("d,rep,m", [(128, 4, 1), (128, 3, 7), (128, 4, 50), (64, 4, 90), (256, 4, 40), (256, 4, 1)])
def test_strided_rows_and_rows_behind_the_last_sequence(d, rep, m):
    H, lens = 2, [77, 140]
    c = R.Cache(K, lens, H, d, 4, 4, 16, "fp16", 16, HALF)
    n, Hq = 2 * m, H * rep
    fused = rand(n + 3, (Hq + 5) * d, dtype=HALF, seed=9)
    q = fused[:, d:(Hq + 1) * d].view(n + 3, Hq, d)
    wide = torch.full((n + 3, (Hq + 2) * d), 7.0, dtype=HALF, device="cuda")
    out = wide[:, d:(Hq + 1) * d].view(n + 3, Hq, d)
    b = c.batch(K, [m, m], total_q=n + 3)
    R.attend(K, c, q, b, out=out)
    assert (wide[n:] == 7).all() and (wide[:, :d] == 7).all() and (wide[:, (Hq + 1) * d:] == 7).all()
    ref, tol = R.attention64(q[:n], *c.sides, c.table.cpu().numpy(), lens, [m, m], c.seed, HALF)
    R.check(out[:n], ref, tol)


@pytest.mark.parametrize("m", [1, 6, 70])
def test_bounds_hold_where_the_tables_break_them(m):
    """seq_lens past max_seq_len and below zero, and more query rows than max_q: clamped, nothing else written."""
    c = R.Cache(K, [90, 90, 90], 2, 128, 4, 4, 16, "fp32", 16, BF16)
    q = rand(3 * m + 2, 8, 128, dtype=BF16, seed=2)
    b = c.batch(K, [m, m, m + 2], lens=[5000, 90, -4], max_q=m, max_seq_len=90)
    out = torch.full_like(q, 5.0)
    R.attend(K, c, q, b, out=out)
    ref, tol = R.attention64(q[:2 * m], *c.sides, c.table.cpu().numpy(), [90, 90], [m, m], c.seed, BF16)
    R.check(out[:2 * m], ref, tol)
    assert (out[2 * m:3 * m] == 0).all() and (out[3 * m:] == 5).all()


@pytest.mark.parametrize("m", [1, 5, 70])
def test_bad_pages_read_nothing_and_are_reported(m):
    c = R.Cache(K, [200, 60], 2, 128, 4, 8, 16, "fp16", 16, HALF)
    good = c.table.clone()
    c.table[0, 3], c.table[0, 7] = 1 << 28, -1
    q = rand(2 * m, 4, 128, dtype=HALF, seed=2)
    out = R.attend(K, c, q, c.batch(K, [m, m]))
    assert K.srftkv_device_fault() == 1 << 17
    assert torch.isfinite(out).all()
    # the other sequence is untouched by it, and rows of zeros stand where the bad pages were
    zero = [p for p in range(c.sides[0].codes.shape[0]) if p not in set(good.flatten().tolist())][:1]
    for p in c.sides:
        p.codes[zero], p.scales[zero] = 0, 0
    table = c.table.cpu().numpy().copy()
    table[0, 3] = table[0, 7] = zero[0]
    ref, tol = R.attention64(q, *c.sides, table, [200, 60], [m, m], c.seed, HALF)
    R.check(out, ref, tol)


@pytest.mark.parametrize("d,m", [(128, 1), (128, 5), (128, 70), (128, 160), (64, 160), (256, 100)])
def test_pages_before_every_window_may_be_gone(d, m):
    """Entries of pages that no query sees are not looked at: nothing is reported, the answer is the same bits."""
    window, lens = 40, [700, 333]
    c = R.Cache(K, lens, 2, d, 4, 4, 16, "fp16", 16, BF16)
    q = rand(2 * m, 8, d, dtype=BF16, seed=2)
    b = c.batch(K, [m, m])
    want = R.attend(K, c, q, b, window=window)
    ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), lens, [m, m], c.seed, BF16, window)
    R.check(want, ref, tol)
    for s, n in enumerate(lens):
        c.table[s, :max(0, n - m - window + 1) // 16] = -1
    assert torch.equal(R.attend(K, c, q, b, window=window), want)
    assert K.srftkv_device_fault() == 0


@pytest.mark.parametrize("d,m", [(128, 170), (64, 170), (256, 110)])
def test_bad_pages_of_long_prompts(d, m):
    """The same where the tiles are laid down before (three row blocks and more)."""
    c = R.Cache(K, [400, 180], 1, d, 4, 8, 16, "e8m0", 32, HALF)
    c.table[0, 3], c.table[0, 7] = 1 << 28, -1
    q = rand(2 * m, 4, d, dtype=HALF, seed=2)
    out = R.attend(K, c, q, c.batch(K, [m, m]))
    assert K.srftkv_device_fault() == 1 << 17
    used = set(c.table.flatten().tolist())
    zero = next(p for p in range(c.sides[0].codes.shape[0]) if p not in used)
    for p in c.sides:
        p.codes[zero], p.scales[zero] = 0, 0
    c.table[0, 3] = c.table[0, 7] = zero
    ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), [400, 180], [m, m], c.seed, HALF)
    R.check(out, ref, tol)


@pytest.mark.parametrize("m", [1, 4, 40, 300])
def test_a_window_of_everything_and_rows_that_see_nothing(m):
    """The largest window equals none, with more query rows than tokens too; a sequence without queries beside it."""
    lens, qlens = [200, 2, 90], [m, m, 0]
    c = R.Cache(K, lens, 1, 128, 8, 8, 16, "fp32", 64, HALF, transform="srft", transform_v="srht", lam=True)
    q = rand(2 * m, 4, 128, dtype=HALF, seed=2)
    b = c.batch(K, qlens)
    want = R.attend(K, c, q, b)
    ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), lens, qlens, c.seed, HALF)
    R.check(want, ref, tol)
    for window in (200, 2**31 - 1):
        assert torch.equal(R.attend(K, c, q, b, window=window), want)
    # and a call of three row blocks none of whose sequences has a query
    b.cu_q.zero_()
    out = torch.full_like(q, 3.0)
    R.attend(K, c, q, b, out=out)
    assert (out == 3).all()


@pytest.mark.parametrize("n", [40, 2500, 12000])
@pytest.mark.parametrize("tr,trv", [("srft", "srht"), ("srht", "srft")])
def test_sides_with_different_transforms(n, tr, trv):
    """bf16 rows of sizes from 2^-30 to 2^30 beside each other, K and V rotated differently; fp32 scales."""
    p = [K.alloc_pages(-(-n // 32), 32, 1, 128, 8, 16, transform=t) for t in (tr, trv)]
    size = torch.exp2(torch.arange(n, device="cuda") % 61 - 30.0)[:, None, None]
    x = [(torch.randn(n, 1, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(s)) * size).bfloat16()
         for s in (1, 2)]
    slots = torch.randperm(n, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    K.srft_kv_quantize_paged(p[0], x[0], p[1], x[1], slots, 9)
    for a, side, t in zip(x, p, (tr, trv)):
        z = O.rotate(R.f64(a), 9, t)
        held = R.held_rows(side, slots.tolist())
        # at most half a step of the group's scale, one eighth of a percent of it for the fp32 arithmetic
        step = np.repeat(np.abs(z).reshape(n, 1, 8, 16).max(-1) / 127, 16, axis=-1)
        assert (np.abs(held - z) <= 0.50125 * step).all()


def test_refusals_on_the_gpu():
    c = R.Cache(K, [500], 1, 128, 4, 4, 16, "fp16", 16, HALF)
    k, v = c.sides
    q, b = rand(1, 4, 128, dtype=HALF), c.batch(K)
    out = torch.full_like(q, 2.0)
    need = K.q4kv_paged_attention_workspace_size(k, 4, b)
    assert need > 0
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    cpu = K.Pages(k.codes.cpu(), k.scales.cpu(), 4, 128, 16, scale_format="fp16")
    for call in (lambda: K.q4kv_paged_attention(q, out, k, v, b, 0.0, 0, 1, ws[:need - 16]),
                 lambda: K.q4kv_paged_attention(q, out, k, v, b, 0.0, 0, 1, None),
                 lambda: K.q4kv_paged_attention(q, out, k, v, b, 0.0, 0, 1, ws[8:]),
                 lambda: K.q4kv_paged_attention(q, out, k, v, b, 0.0, 0, 1, ws.cpu()),
                 lambda: K.q4kv_paged_attention(q, out, cpu, cpu, b, 0.0, 0, 1, ws),
                 lambda: K.q4kv_paged_attention(q, out, k, cpu, b, 0.0, 0, 1, ws),
                 lambda: K.srft_kv_quantize_paged(cpu, q[:, :1].cpu(), None, None, c.slots[:1].cpu(), 1),
                 lambda: K.srft_kv_quantize_paged(k, q[:, :1], None, None, c.slots[:1].cpu(), 1),
                 lambda: K.srft_kv_quantize_paged(k, None, v, q[:, :1], c.slots[:1], 1)):
        with pytest.raises(K.SrftKvError) as e:
            call()
        assert e.value.code == K.SRFTKV_ERR_INVALID
    assert (out == 2).all()
    one = c.batch(K, max_seq_len=100)  # one split: no workspace
    assert K.q4kv_paged_attention_workspace_size(k, 4, one) == 0
    K.q4kv_paged_attention(q, out, k, v, one, 0.0, 0, 1, None)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("m", [1, 4, 80])
@pytest.mark.parametrize("fmt", ["fp32", "fp16", "e8m0"])
def test_ranges_of_the_scales(m, fmt):
    """Rows of size 2^9 beside rows of size 2^-10: within the range the header states, K's and V's alike."""
    lens = [150, 70]
    c = R.Cache(K, lens, 1, 128, 8, 8, 16, fmt, 16, BF16, gain=1.0)
    for p, x in zip(c.sides, c.rows):
        x[::3] *= 2.0**-10
    c.rows[1][1::3] *= 2.0**9
    K.srft_kv_quantize_paged(c.sides[0], c.rows[0], c.sides[1], c.rows[1], c.slots, c.seed)
    q = rand(2 * m, 4, 128, dtype=BF16, seed=2)
    out = R.attend(K, c, q, c.batch(K, [m, m]))
    ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), lens, [m, m], c.seed, BF16)
    R.check(out, ref, tol + 2.0**-24)


# ---------------------------------------------------------------------------
# Used together, and the ways a program calls it
# ---------------------------------------------------------------------------
def test_a_conversation():
    """A prompt in chunks, then single tokens and a drafted run, each written and attended: every step against the
    definition over the rows the pools hold by then."""
    H, rep, d, page, lens = 2, 3, 128, 16, [150, 41]
    c = R.Cache(K, lens, H, d, 8, 4, 16, "fp16", page, BF16)
    for i, p in enumerate(c.sides):
        R.garbage(p, 8 + i)
    at = [0, 0]
    for step in ([60, 20], [70, 9], [1, 1], [1, 1], [4, 5], [1, 0], [13, 5]):
        spans = [(b, at[b], at[b] + m) for b, m in enumerate(step)]
        first = [0, lens[0]]
        idx = torch.cat([torch.arange(first[b] + lo, first[b] + hi, device="cuda") for b, lo, hi in spans])
        K.srft_kv_quantize_paged(c.sides[0], c.rows[0][idx], c.sides[1], c.rows[1][idx], c.slots_of(spans), c.seed)
        at = [a + m for a, m in zip(at, step)]
        q = rand(sum(step), H * rep, d, dtype=BF16, seed=sum(at))
        out = R.attend(K, c, q, c.batch(K, step, lens=at))
        ref, tol = R.attention64(q, *c.sides, c.table.cpu().numpy(), at, step, c.seed, BF16)
        R.check(out, ref, tol)
    y = [torch.empty_like(r) for r in c.rows]
    K.srft_kv_dequantize_paged(c.sides[0], y[0], c.sides[1], y[1], c.slots, c.seed)
    for p, got in zip(c.sides, y):
        z = R.held_rows(p, c.slots.cpu().numpy())
        want = O.unrotate(z, c.seed)
        assert np.all(np.abs(R.f64(got) - want) <= R.dequant_tolerance(z, 1.0, want, BF16))


@pytest.mark.parametrize("m,rep", [(1, 4), (5, 4), (90, 4), (160, 4)])
def test_captured_and_replayed(m, rep):
    """A captured step (write, then attention) replayed with other rows, lengths and tables equals the eager calls
    bit for bit; two runs of one call are the same bits."""
    H, d = 2, 128
    c = R.Cache(K, [700, 300], H, d, 4, 4, 16, "fp16", 16, BF16)
    q = rand(2 * m, H * rep, d, dtype=BF16, seed=1)
    xk, xv = rand(2 * m, H, d, dtype=BF16, seed=2), rand(2 * m, H, d, dtype=BF16, seed=3)
    slots = c.slots_of([(0, 700 - m, 700), (1, 300 - m, 300)])
    batch = c.batch(K, [m, m])
    k, v = c.sides
    ws = torch.empty(max(16, K.q4kv_paged_attention_workspace_size(k, H * rep, batch)), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)

    def step():
        K.srft_kv_quantize_paged(k, xk, v, xv, slots, c.seed)
        K.q4kv_paged_attention(q, out, k, v, batch, 0.0, 0, c.seed, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for it, lens in enumerate(([700, 300], [650, 299], [m, 17 + m], [333, 1])):
        q.copy_(rand(*q.shape, dtype=BF16, seed=10 + it))
        xk.copy_(rand(*xk.shape, dtype=BF16, seed=20 + it))
        batch.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        slots.copy_(torch.cat([c.slots_of([(0, max(0, lens[0] - m), max(0, lens[0] - m) + m)]),
                               c.slots_of([(1, max(0, lens[1] - m), max(0, lens[1] - m) + m)])]))
        graph.replay()
        got = out.clone()
        ws.fill_(0xFF)  # a workspace's old contents do not matter
        step()
        assert torch.equal(got, out)
        step()
        assert torch.equal(got, out)


FIRST_CALLS = """
import torch, int8_kv_cache_srft_gb300 as K
k, v = [K.alloc_pages(64, 16, 2, 128, 4, 16) for _ in range(2)]
for p in (k, v):
    p.codes.fill_(0x11), p.scales.fill_(0.5)
table = torch.arange(64, dtype=torch.int32, device="cuda").view(1, 64)
for m in (1, 6, 40, 200):
    cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
    b = K.PagedBatch(table, torch.tensor([900], dtype=torch.int32, device="cuda"), cu, total_q=m, max_q=m)
    q, x = torch.randn(m, 8, 128, device="cuda").half(), torch.randn(m, 2, 128, device="cuda").half()
    out, slots = torch.empty_like(q), torch.arange(900 - m, 900, device="cuda")
    ws = torch.empty(max(16, K.q4kv_paged_attention_workspace_size(k, 8, b)), dtype=torch.uint8, device="cuda")
    def step():
        K.srft_kv_quantize_paged(k, x, v, x, slots, 1)
        K.q4kv_paged_attention(q, out, k, v, b, 0.0, 0, 1, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    got = out.clone()
    step()
    assert torch.equal(got, out), m
assert K.srftkv_device_fault() == 0
"""


def test_the_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_streams_at_once():
    c = [R.Cache(K, [900, 200], 2, 128, 4, 4, 16, "fp32", 16, HALF, data_seed=s) for s in (1, 2)]
    q = [rand(2, 8, 128, dtype=HALF, seed=s) for s in (3, 4)]
    b = [x.batch(K) for x in c]
    want = [R.attend(K, x, y, z) for x, y, z in zip(c, q, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in c]
    outs = []
    for _ in range(20):
        for x, y, z, s in zip(c, q, b, streams):
            with torch.cuda.stream(s):
                outs.append(R.attend(K, x, y, z))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, want[i % 2])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_large_calls_on_two_streams_at_once(d):
    """Prompts on one stream beside a large write and read on the other: the same bits as one after the other."""
    H, n = 2, 16000
    c = R.Cache(K, [900, 400], H, d, 4, 4, 16, "fp16", 16, BF16)
    q, b = rand(1300, 4 * H, d, dtype=BF16, seed=3), c.batch(K, [900, 400])
    want = R.attend(K, c, q, b)
    pools = [K.alloc_pages(n // 32, 32, H, d, 8, 16, scale_format="e8m0") for _ in range(2)]
    x = [rand(n, H, d, dtype=BF16, seed=s) for s in (5, 6)]
    y = [torch.zeros_like(a) for a in x]
    slots = torch.randperm(n, device="cuda")

    def codec():
        K.srft_kv_quantize_paged(pools[0], x[0], pools[1], x[1], slots, 7)
        K.srft_kv_dequantize_paged(pools[0], y[0], pools[1], y[1], slots, 7)

    codec()
    torch.cuda.synchronize()
    kept = [a.clone() for a in y] + [p.codes.clone() for p in pools]
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for a in y + [p.codes for p in pools]:
        a.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            outs.append(R.attend(K, c, q, b))
        with torch.cuda.stream(streams[1]):
            codec()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    assert all(torch.equal(a, k) for a, k in zip(y + [p.codes for p in pools], kept))


def test_stream_argument():
    """Work goes to the stream given, not the current one."""
    c = R.Cache(K, [100], 1, 64, 4, 4, 16, "fp32", 16, HALF)
    q = rand(1, 2, 64, dtype=HALF)
    want = R.attend(K, c, q, c.batch(K))
    torch.cuda.synchronize()
    s, out, b = torch.cuda.Stream(), torch.zeros_like(q), c.batch(K)
    ws = torch.empty(max(16, K.q4kv_paged_attention_workspace_size(c.sides[0], 2, b)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    K.q4kv_paged_attention(q, out, *c.sides, b, 0.0, 0, c.seed, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes: its last pages are written, read back and attended."""
    H, d, page, n_pages = 8, 256, 256, 9000
    p = [K.alloc_pages(n_pages, page, H, d, 8, 256, scale_format="e8m0") for _ in range(2)]
    assert p[0].codes.numel() > 1 << 32
    lens = [300]
    table = torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda")
    t = torch.arange(300, device="cuda")
    slots = table[0, t // page].long() * page + t % page
    x = [rand(300, H, d, dtype=BF16, seed=s) for s in (1, 2)]
    K.srft_kv_quantize_paged(p[0], x[0], p[1], x[1], slots, 3)
    y = [torch.empty_like(a) for a in x]
    K.srft_kv_dequantize_paged(p[0], y[0], p[1], y[1], slots, 3)
    for a, b in zip(x, y):
        assert (a.float() - b.float()).abs().max() < 0.2
    for m in (1, 30):
        q = rand(m, H, d, dtype=BF16, seed=7)
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        b = K.PagedBatch(table, torch.tensor(lens, dtype=torch.int32, device="cuda"), cu, total_q=m, max_q=m)
        ws = torch.empty(max(16, K.q4kv_paged_attention_workspace_size(p[0], H, b)), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(q)
        K.q4kv_paged_attention(q, out, p[0], p[1], b, 0.0, 0, 3, ws)
        # over the rows read back (their output rounding adds to the tolerance: 2^-8 of a score of size sqrt(d))
        k, v = y[0].double(), y[1].double()
        s = torch.einsum("mhd,thd->hmt", q.double(), k) / d**0.5
        s.masked_fill_(torch.arange(300, device="cuda") > torch.arange(300 - m, 300, device="cuda")[:, None], -np.inf)
        want = torch.einsum("hmt,thd->mhd", s.softmax(-1), v)
        assert (out.double() - want).abs().max() < 0.02
