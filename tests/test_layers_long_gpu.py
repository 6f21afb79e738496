"""Paged attention where a CTA walks many tiles of a row, or a row is cut into
many pieces, against the definition in 64 bits on the device: o, lse and the
weights drawn.

Bounds, per element, before any run.  With u = 2^-23 (unit of the fp32 sums: the
tensor cores may truncate where an FMA rounds):
  a score is a d-term sum, off by at most e = scale (d + 4) u max |q| |k|, and
  the argument of exp2 (score minus reference) is rounded: top u each, top the
  largest |score|;
  the weights of a row are summed in tiles of at most 64 tokens (four chains or
  fewer: counted as 64 terms), over the tiles of a CTA, then over its pieces:
  m = 64 + tiles + pieces terms one after another, not the row's length;
  so a weight is off, relative to itself, by rel = 2 e + 2 top u + m u + 2^-20
  (exp2 is within 2 ulp; the division), and with bf16 also by P's rounding, 2^-8;
  o sums the same way (m u more):
  |o - ref| <= sum p|v| (rel + m u + 2^-8) + half a step of o,
  |lse - ref| <= rel + |lse| 2^-22,
  |drawn - ref| <= drawn (rel + rows u) + 2^-23 |mass|.
tests/test_layers_long_bounds_cpu.py holds these bounds against mistakes: one
tile of 64 of 70001 tokens left out, taken twice or taken from its neighbour's
place is seen.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


def build(gen, lengths, H, page, d, dtype, bad=()):
    """Pools with scattered pages, NaN where no token lies; bad: (request,
    table entry) pairs whose page number is out of range."""
    R = len(lengths)
    row_pages = -(-max(lengths) // page)
    pages = R * row_pages + 1
    k, v = (torch.randn((pages, H, page, d), generator=gen, device=gen.device).to(dtype) for _ in range(2))
    table = torch.randperm(pages, generator=gen, device=gen.device)[:R * row_pages].to(torch.int32).reshape(R, row_pages)
    for r, n in enumerate(lengths):
        for e in range(n // page, row_pages):
            at = max(0, n - e * page)
            k[table[r, e].long(), :, at:] = float("nan")
            v[table[r, e].long(), :, at:] = float("nan")
    shown = table.clone()
    for r, e in bad:
        shown[r, e] = pages + 5
    return k, v, table, shown


def reference(q, k, v, table, shown, lengths, scale, mass, keep=None):
    """o, lse, drawn + mass, sum p|v| and the largest |score| in 64 bits.  keep
    (mistakes planted by the tests of the bounds): what becomes of the positions."""
    R, W, H_q, d = q.shape
    pages, H, page, _ = k.shape
    G, dev = H_q // H, q.device
    o, spread = (torch.zeros(R, W, H_q, d, dtype=torch.float64, device=dev) for _ in range(2))
    lse = torch.full((R, W, H_q), -float("inf"), dtype=torch.float64, device=dev)
    drawn = mass.double().clone()
    top = 0.0
    for r, n in enumerate(lengths):
        j = torch.arange(n, device=dev)
        if keep is not None:
            j = keep(j)
        entry = shown[r].long()[j // page]
        live = (entry >= 0) & (entry < pages)
        j = j[live]
        if not len(j):
            continue
        at = table[r].long()[j // page]
        for h in range(H):
            kk, vv = k[at, h, j % page].double(), v[at, h, j % page].double()
            qq = q[r, :, h * G:(h + 1) * G].double()
            s = torch.einsum("wgd,nd->wgn", qq, kk) * scale
            top = max(top, float(s.abs().max()))
            l = torch.logsumexp(s, -1)
            p = torch.exp(s - l[..., None])
            o[r, :, h * G:(h + 1) * G] = torch.einsum("wgn,nd->wgd", p, vv)
            spread[r, :, h * G:(h + 1) * G] = torch.einsum("wgn,nd->wgd", p, vv.abs())
            lse[r, :, h * G:(h + 1) * G] = l
            drawn[r, h].index_add_(0, j, p.sum((0, 1)))
    return o, lse, drawn, spread, top


def bounds(q, k, scale, tiles, pieces, ref, mass):
    """Bounds of o, lse and the weights drawn (the module's text), from the reference."""
    ro, rl, rm, spread, top = ref
    d, rows = q.shape[3], q.shape[1] * q.shape[2] // k.shape[1]
    qn = float(q.double().square().sum(-1).max().sqrt())
    kn = float(torch.nan_to_num(k.double(), nan=0.0).square().sum(-1).max().sqrt())
    m = 64 + tiles + pieces
    rel = 2 * scale * (d + 4) * U * qn * kn + 2 * top * U + m * U + 2.0 ** -20
    bf, half = (2.0 ** -8, 2.0 ** -8) if q.dtype == torch.bfloat16 else (0.0, 2.0 ** -24)
    return (1.01 * (spread * (rel + m * U + bf) + half * ro.abs()) + 1e-30, rel + rl.abs() * 2.0 ** -22,
            1.01 * (rm - mass.double()) * (rel + rows * U) + rm * 2.0 ** -23)


def check(q, k, v, table, shown, lengths, tiles, pieces, kernel=0, scale=None):
    import linear_attention_beam_shared_b200 as L
    R, W, H_q, d = q.shape
    H, page = k.shape[1:3]
    scale = d ** -0.5 if scale is None else scale
    mass = torch.rand((R, H, table.shape[1] * page), device="cuda")
    mass_out = torch.full_like(mass, -3.0)
    lse = torch.full((R, W, H_q), 7.0, device="cuda")
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o = L.onela_paged_attention(q, k, v, shown, n, scale=scale, mass=mass, mass_out=mass_out, lse=lse, kernel=kernel)
    ref = reference(q, k, v, table, shown, lengths, scale, mass)
    lims = bounds(q, k, scale, tiles, pieces, ref, mass)
    assert bool((torch.isneginf(lse) == torch.isneginf(ref[1])).all())
    for name, got, want, lim in zip(("o", "lse", "weights"), (o, lse, mass_out), ref, lims):
        if name == "weights":
            past = torch.arange(mass.shape[2], device="cuda")[None, None] >= n[:, None, None]
            assert bool((got[past.expand_as(got)] == -3.0).all())
            got = torch.where(past, mass, got)
        over = torch.where(torch.isneginf(want), 0.0, (got.double() - want).abs() / lim.clamp_min(1e-300))
        assert bool((over <= 1).all()), f"{name}: {float(over.max())} of its bound"
    return o, lse, mass_out


# One part per head (148 key-value heads fill the SMs), so a CTA walks the whole
# row: 17, 35 or 58 tiles of 64, the last one not full.
@pytest.mark.parametrize("page", [8, 16, 20])
@pytest.mark.parametrize("W,G,d", [(20, 1, 64), (11, 6, 128), (64, 4, 64), (75, 4, 128), (5, 8, 256)])
@pytest.mark.parametrize("tiles,left", [(17, 5), (35, 63), (58, 1)])
def test_a_partly_filled_tile_behind_many_full_ones(tiles, left, W, G, d, page):
    """The last tokens carry the weight: K's rows there lie along the queries'
    common direction, so a score of other rows shows."""
    gen = torch.Generator(device="cuda").manual_seed(tiles * W + page)
    H, n = 148, 64 * (tiles - 1) + left
    k, v, table, shown = build(gen, [n], H, page, d, torch.bfloat16)
    u = torch.sign(torch.randn((H, d), generator=gen, device="cuda"))
    q = (torch.randn((1, W, H, G, d), generator=gen, device="cuda") * 0.5 + u[None, None, :, None]).reshape(1, W, H * G, d).bfloat16()
    last = torch.arange(n - left, n, device="cuda")
    at = table[0].long()[last // page]
    boost = 6.0 * d ** -0.5  # adds 6 to these tokens' scores
    k[at, :, last % page] = (k[at, :, last % page].float() + boost * u).bfloat16()
    check(q, k, v, table, shown, [n], tiles, 1)


@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("W,G,d", [(20, 1, 64), (64, 4, 128)])
def test_a_bad_page_behind_many_full_tiles(W, G, d, page):
    """Tiles 20 and 40 of 50 miss a page's tokens."""
    gen = torch.Generator(device="cuda").manual_seed(W + page)
    H, n = 148, 64 * 50
    k, v, table, shown = build(gen, [n], H, page, d, torch.bfloat16, bad=[(0, 20 * 64 // page + 1), (0, 40 * 64 // page)])
    q = torch.randn((1, W, H * G, d), generator=gen, device="cuda").bfloat16()
    check(q, k, v, table, shown, [n], 50, 1)


@pytest.mark.parametrize("lengths,W,H_q,H,d,tiles,pieces", [
    ([65541], 32, 32, 8, 128, 57, 19), ([4999] * 8, 8, 32, 8, 128, 40, 4), ([4990 + 3 * r for r in range(9)], 16, 16, 8, 64, 40, 4),
    ([9000, 70, 1, 12000, 0, 333], 70, 8, 4, 128, 40, 37)])
def test_parts_that_cross_requests(lengths, W, H_q, H, d, tiles, pieces):
    """Parts of many tiles that end inside a request, begin inside the next,
    and meet partly filled tiles on the way."""
    gen = torch.Generator(device="cuda").manual_seed(len(lengths))
    k, v, table, shown = build(gen, lengths, H, 16, d, torch.bfloat16)
    q = torch.randn((len(lengths), W, H_q, d), generator=gen, device="cuda").bfloat16()
    check(q, k, v, table, shown, lengths, tiles, pieces)


@pytest.mark.parametrize("W,pad", [(1, 3), (40, 3), (40, 8), (40, 1)])
def test_one_scratch_buffer_for_a_slice_of_a_projection(W, pad):
    """q as a slice of a projection whose token stride is or is not a multiple
    of 8: the call takes the buffer that was sized for that stride."""
    import linear_attention_beam_shared_b200 as L
    gen = torch.Generator(device="cuda").manual_seed(W + pad)
    H, G, d, page, n = 2, 4, 64, 16, 700
    k, v, table, shown = build(gen, [n], H, page, d, torch.bfloat16)
    stride = H * G * d + pad
    wide = torch.randn((1, W, stride), generator=gen, device="cuda").bfloat16()
    q = wide[:, :, :H * G * d].unflatten(-1, (H * G, d))
    need = L.onela_paged_attention_scratch_bytes(1, W, H * G, H, d, "bf16", page, k.shape[0], table.shape[1], want_mass=True,
                                                 q_stride=stride)
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = [torch.zeros((1, H, table.shape[1] * page), device="cuda") for _ in range(2)]
    a = L.onela_paged_attention(q, k, v, table, lengths, mass_out=out[0], scratch=scratch)
    b = L.onela_paged_attention(q, k, v, table, lengths, mass_out=out[1])
    assert torch.equal(a, b) and torch.equal(*out)
    check(q, k, v, table, shown, [n], 11, 11)
    with pytest.raises(L.OnelaError):
        L.onela_paged_attention(q, k, v, table, lengths, mass_out=out[0], scratch=scratch[:need - 256])


@pytest.mark.parametrize("times", [1.0, 1.7109375, 1.3046875])
@pytest.mark.parametrize("power", [20, 34, 60, 100])
@pytest.mark.parametrize("kind", ["all_low", "first_low", "one_high"])
@pytest.mark.parametrize("W,d,kernel", [(1, 64, 0), (3, 128, 0), (1, 256, 0), (40, 64, 0), (90, 128, 0), (40, 256, 0), (5, 64, 1)])
def test_scores_far_from_zero(W, d, kernel, kind, power, times):
    """Scores of 2^power and more, as a fill for tokens that are not to count
    gives them: the softmax is of differences, so the scores' size alone loses
    nothing.  q and K are signs times one number, every product q k is exact and
    equal ones are equal (with `times` the scaled score is not exact), so the weights are those of a few cases: one over the
    number of tokens that share the largest score, 0 elsewhere (2^-28000 and less)."""
    import linear_attention_beam_shared_b200 as L
    H, G, page, n = 2, 4, 16, 64 * 9 + 21
    gen = torch.Generator(device="cuda").manual_seed(W + d)
    k, v, table, _ = build(gen, [n], H, page, d, torch.bfloat16)
    u = torch.sign(torch.randn((H, d), generator=gen, device="cuda"))
    q = u[None, None, :, None].expand(1, W, H, G, d).reshape(1, W, H * G, d).bfloat16().contiguous()
    j = torch.arange(n, device="cuda")
    size = torch.zeros(n, device="cuda")
    if kind == "all_low":
        size[:] = -times * 2.0 ** power
    elif kind == "first_low":
        size[:200] = -times * 2.0 ** power
    else:
        size[311] = times * 2.0 ** power
    k[table[0].long()[j // page], :, j % page] = (size[:, None, None] * u).bfloat16()
    top = size == size.max()
    m = int(top.sum())
    vv = v[table[0].long()[j // page], :, j % page].double()[top].mean(0)           # [H][d]
    spread = v[table[0].long()[j // page], :, j % page].double()[top].abs().mean(0)
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    mass_out = torch.full((1, H, table.shape[1] * page), -3.0, device="cuda")
    lse = torch.empty((1, W, H * G), device="cuda")
    o = L.onela_paged_attention(q, k, v, table, lengths, lse=lse, mass_out=mass_out, kernel=kernel)
    ref = vv[None, None, :, None].expand(1, W, H, G, d).reshape(o.shape)
    lim = 2.0 ** -8 * ref.abs() + ((2.0 ** -8 + 200 * U) * spread)[None, None, :, None].expand(1, W, H, G, d).reshape(o.shape)
    assert bool(((o.double() - ref).abs() <= 1.01 * lim).all())
    s = float(size.max()) * d * d ** -0.5 + float(torch.tensor(float(m)).log())
    assert bool(((lse.double() - s).abs() <= abs(s) * 2.0 ** -22 + 1e-5).all())
    want = torch.where(top, torch.full((n,), W * G / m, device="cuda", dtype=torch.float64), torch.zeros(n, device="cuda", dtype=torch.float64))
    assert bool(((mass_out[0, :, :n].double() - want).abs() <= want * (200 + W * G) * U + 1e-30).all())


# The division gives a row of 1094 tiles of 64 to at most 3 CTAs an SM over 2
# heads, 222 parts (narrow; 74 with d = 256), 148 / 2 or fewer (wide), or 2188 tiles
# of 32 to 4 an SM, 296 parts (general): 300 pieces, and at most 60 tiles and warps'
# sums in one.
@pytest.mark.parametrize("W,H_q,d,dtype,kernel", [
    (1, 8, 128, "bf16", 0), (1, 8, 64, "bf16", 0), (1, 8, 256, "bf16", 0), (1, 8, 128, "bf16", 1), (24, 8, 128, "bf16", 0),
    (24, 8, 256, "bf16", 0), (90, 8, 64, "bf16", 0), (1, 8, 128, "f32", 0), (3, 4, 80, "f32", 0)])
def test_a_row_cut_into_many_pieces(W, H_q, d, dtype, kernel):
    gen = torch.Generator(device="cuda").manual_seed(W + d)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    k, v, table, shown = build(gen, [70001], 2, 64, d, dt)
    q = torch.randn((1, W, H_q, d), generator=gen, device="cuda").to(dt)
    check(q, k, v, table, shown, [70001], 60, 300, kernel=kernel)
