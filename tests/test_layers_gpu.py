"""GPU parity of the operators around a GDN layer against the fp64 oracle
(oracle/layers.py), through the public entry points.

Tolerances are worked out per element, never looked up from a run.  With u the
unit of the fp32 sums (2^-23: the tensor cores may truncate where an FMA
rounds) and n the number of attended tokens:
  a score is a d-term sum, off by at most e = scale * (d + 4) * u * max_j
  sum_i |q_i k_ij|; a weight p = exp(s - max) / sum is off, relative to itself, by at most
  2 e + n u + 2^-20 (the argument of exp2 is rounded: 2^-23 per unit of score,
  scores below 8 here; exp2 itself 2 ulp; the division); with bf16 inputs each weight may
  also be rounded to bf16 (2^-8) on its way into the tensor cores; o sums n
  terms p v more (n u).  So |o - ref| <= spread * rel + half a step of o, with
  spread = sum p |v|.
"""
import numpy as np
import pytest
import torch

from oracle import layers

pytestmark = pytest.mark.gpu

U = 2.0 ** -23
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def f64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """Pools with scattered pages; slots past a row's length hold NaN."""

    def __init__(self, rng, lengths, H, page, d, dtype, row_pages=None, spare=3):
        R = len(lengths)
        need = max(1, -(-max(lengths) // page))
        self.row_pages = row_pages or need + 1
        pages = R * self.row_pages + spare
        k, v = (rng.standard_normal((pages, H, page, d)).astype(np.float32) for _ in range(2))
        self.table = rng.permutation(pages)[:R * self.row_pages].reshape(R, self.row_pages).astype(np.int32)
        used = np.zeros((pages, page), bool)
        for r, n in enumerate(lengths):
            for p in range(n):
                used[self.table[r, p // page], p % page] = True
        hole = ~used[:, None, :, None]
        k, v = np.where(hole, np.nan, k), np.where(hole, np.inf, v)
        self.k, self.v = (torch.from_numpy(x).to(DT[dtype]).cuda() for x in (k, v))
        self.lengths = np.array(lengths, np.int32)

    def dev(self):
        return self.k, self.v, torch.from_numpy(self.table).cuda(), torch.from_numpy(self.lengths).cuda()

    def host(self):
        return f64(self.k), f64(self.v), self.table, self.lengths


def draw_beam(rng, R, W, H, d, dtype, blen, page=1):
    """A beam pool whose tables share entries (ancestors); blen [R][W]."""
    rows = max(1, -(-int(np.max(blen)) // page))
    pages = max(4, R * W * rows // 2)
    k, v = (torch.from_numpy(rng.standard_normal((pages, H, page, d)).astype(np.float32)).to(DT[dtype]).cuda()
            for _ in range(2))
    table = rng.integers(0, pages, (R, W, rows)).astype(np.int32)
    return k, v, table, np.asarray(blen, np.int32)


def check_attention(q, cache, beam=None, scale=None, mass=None, kernel=0, with_lse=True, dtype="bf16", status=None):
    import linear_attention_beam_shared_b200 as L
    R, W, H_q, d = q.shape
    k, v, table, lengths = cache.dev()
    bdev = None if beam is None else (beam[0], beam[1], torch.from_numpy(beam[2]).cuda(), torch.from_numpy(beam[3]).cuda())
    lse = torch.full((R, W, H_q), 7.0, device="cuda") if with_lse else None
    m_in = None if mass is None else torch.from_numpy(mass).cuda()
    m_out = None if mass is None else torch.full_like(m_in, -3.0)
    o = L.onela_paged_attention(q, k, v, table, lengths, beam=bdev, scale=scale, mass=m_in, mass_out=m_out, lse=lse,
                                kernel=kernel, status=status)
    hbeam = None if beam is None else (f64(beam[0]), f64(beam[1]), beam[2], beam[3])
    ro, rl, rm, spread = layers.paged_attention(f64(q), *cache.host(), beam=hbeam, scale=scale, mass=mass)
    sc = d ** -0.5 if scale is None else scale
    n = int(np.max(np.clip(cache.lengths, 0, None), initial=0)) + (0 if beam is None else int(beam[3].max()))
    qn, kn = np.abs(f64(q)).max(), max(np.nanmax(np.abs(f64(cache.k)), initial=0.0), 0 if beam is None else np.abs(f64(beam[0])).max())
    # max_j sum_i |q_i k_ij| <= |q| |k| (Cauchy-Schwarz), norms of d entries.
    cs = min(d * qn * kn, np.sqrt((f64(q) ** 2).sum(-1).max()) * np.sqrt(d) * kn)
    e = sc * (d + 4) * U * cs
    top = sc * cs
    rel = 2 * e + 2 * n * U + 2.0 ** -20 + 2 * top * U
    bf = 2.0 ** -8 if dtype == "bf16" else 0.0
    err = np.abs(f64(o) - ro)
    lim = spread * (rel + bf) * 1.01 + HALF[dtype] * np.abs(ro) * 1.01
    assert np.isfinite(f64(o)).all()
    assert (err <= lim + 1e-30).all(), f"o off by {(err - lim).max()} at {np.unravel_index((err - lim).argmax(), err.shape)}"
    if with_lse:
        g = f64(lse)
        assert (np.isneginf(g) == np.isneginf(rl)).all()
        fin = np.isfinite(rl)
        assert (np.abs(g[fin] - rl[fin]) <= rel + np.abs(rl[fin]) * 2.0 ** -22).all()
    if mass is not None:
        g = f64(m_out)
        for r in range(R):
            ln = layers.clamp(cache.lengths[r], g.shape[2])
            assert (g[r, :, ln:] == -3.0).all()
            a, b = g[r, :, :ln], rm[r, :, :ln]
            drawn = b - mass[r, :, :ln]
            M = W * H_q // cache.k.shape[1]
            assert (np.abs(a - b) <= drawn * (rel + M * U) * 1.01 + np.abs(b) * 2.0 ** -23).all()
    return o


def rand_q(rng, R, W, H, d, dtype):
    return torch.from_numpy(rng.standard_normal((R, W, H, d)).astype(np.float32)).to(DT[dtype]).cuda()


SHAPES = [
    # R, W, H_q, H_kv, d, lengths, page
    (1, 1, 1, 1, 64, [1], 16),
    (1, 1, 4, 4, 128, [129], 16),
    (3, 1, 16, 4, 128, [0, 257, 40], 16),
    (2, 1, 8, 1, 256, [700, 33], 64),
    (5, 1, 6, 2, 64, [1, 15, 16, 17, 300], 8),
    (2, 1, 16, 1, 128, [95, 1000], 1),
    (1, 1, 24, 1, 64, [450], 24),
    (2, 1, 6, 2, 80, [77, 300], 16),
    (1, 1, 3, 3, 37, [140], 5),
    (2, 2, 4, 2, 1, [140, 3], 5),
    (1, 5, 8, 4, 128, [260], 16),
    (2, 33, 8, 2, 64, [200, 0], 16),
    (1, 70, 4, 2, 256, [500], 32),
    (2, 64, 8, 2, 128, [513, 127], 16),
    (1, 129, 4, 4, 128, [385], 48),
    (1, 20, 8, 2, 128, [333], 8),
    (1, 20, 8, 2, 64, [333], 24),
    (2, 40, 8, 2, 128, [200, 90], 40),
    (1, 40, 8, 2, 128, [200], 1),
    (1, 24, 8, 2, 256, [150], 20),
    (1, 17, 1, 1, 128, [5000], 16),
    (3, 4, 8, 2, 256, [65, 64, 63], 16),
    (1, 300, 4, 2, 64, [129], 512),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:5])) + f"-p{s[6]}")
def test_attention_matches_oracle(shape, dtype):
    R, W, H_q, H_kv, d, lengths, page = shape
    rng = np.random.default_rng(R * 7 + W * 11 + d + page)
    check_attention(rand_q(rng, R, W, H_q, d, dtype), Cache(rng, lengths, H_kv, page, d, dtype), dtype=dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,W,H_q,H_kv,d,lengths,page,bmax,bpage", [
    (1, 1, 4, 2, 64, [50], 16, 3, 1), (2, 7, 8, 2, 128, [0, 300], 16, 7, 1), (1, 40, 8, 4, 64, [700], 32, 12, 4),
    (2, 65, 4, 1, 256, [129, 64], 16, 5, 1), (1, 2, 2, 1, 30, [9], 3, 40, 8)])
def test_attention_with_beam_tokens_and_mass(R, W, H_q, H_kv, d, lengths, page, bmax, bpage, dtype):
    rng = np.random.default_rng(W + d)
    blen = rng.integers(0, bmax + 1, (R, W))
    blen[0, 0] = bmax
    if W > 1:
        blen[:, 1] = 0  # with no prompt either, a row with nothing at all
    cache = Cache(rng, lengths, H_kv, page, d, dtype)
    mass = rng.random((R, H_kv, cache.row_pages * page)).astype(np.float32)
    check_attention(rand_q(rng, R, W, H_q, d, dtype), cache, beam=draw_beam(rng, R, W, H_kv, d, dtype, blen, bpage),
                    mass=mass, scale=0.3, dtype=dtype)


@pytest.mark.parametrize("W,H_q,H_kv,d,dtype", [(1, 8, 2, 128, "bf16"), (40, 8, 2, 128, "bf16"), (3, 4, 2, 48, "f32")])
def test_mass_alone_is_written_in_place_and_sums_to_the_rows(W, H_q, H_kv, d, dtype):
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(3)
    cache = Cache(rng, [333, 0], H_kv, 16, d, dtype)
    q = rand_q(rng, 2, W, H_q, d, dtype)
    k, v, table, lengths = cache.dev()
    m = torch.zeros((2, H_kv, cache.row_pages * 16), device="cuda")
    L.onela_paged_attention(q, k, v, table, lengths, mass_out=m)
    rows = W * H_q // H_kv
    # Each row's weights sum to 1 up to the relative error of a weight.
    assert np.abs(f64(m)[0].sum(-1) - rows).max() <= rows * (1e-4)
    once = m.clone()
    L.onela_paged_attention(q, k, v, table, lengths, mass=m, mass_out=m)
    np.testing.assert_allclose(f64(m), 2 * f64(once), rtol=2.0 ** -22)


@pytest.mark.parametrize("kernel", [1, 0])
def test_attention_peaked_and_shifted_scores(kernel):
    """Scores in the hundreds: the softmax must not leave the range of exp."""
    rng = np.random.default_rng(8)
    for W in (1, 70):
        cache = Cache(rng, [400], 2, 16, 64, "bf16")
        q = rand_q(rng, 1, W, 4, 64, "bf16") * 40
        check_attention(q, cache, kernel=kernel)


def test_attention_query_slice_of_a_projection():
    rng = np.random.default_rng(9)
    for W in (1, 40):
        wide = rand_q(rng, 2, W, 12, 128, "bf16")
        check_attention(wide[:, :, :8], Cache(rng, [100, 300], 2, 16, 128, "bf16"))
        check_attention(wide[:, :, 4:], Cache(rng, [100, 300], 2, 16, 128, "bf16"))


@pytest.mark.parametrize("W", [1, 40])
def test_attention_bad_pages_and_lengths_are_left_out(W):
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(10)
    cache = Cache(rng, [100, 60, 30], 2, 16, 64, "bf16", row_pages=8)
    cache.table[0, 2], cache.table[1, 0] = -1, 10 ** 6
    beam = draw_beam(rng, 3, W, 2, 64, "bf16", np.full((3, W), 4))
    beam[2][0, 0, 1], beam[2][2, 0, 3] = -5, 2 ** 30
    cache.lengths[2] = -4
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    check_attention(rand_q(rng, 3, W, 4, 64, "bf16"), cache, beam=beam, status=status,
                    mass=np.zeros((3, 2, 128), np.float32))
    assert status.item() == L.ONELA_STATUS_PAGE | L.ONELA_STATUS_LENGTH
    # A length past the row: the row's tokens, and the bit.
    full = Cache(rng, [32], 1, 16, 64, "bf16", row_pages=2)
    full.lengths[0] = 40
    status.zero_()
    check_attention(rand_q(rng, 1, W, 1, 64, "bf16"), full, status=status)
    assert status.item() == L.ONELA_STATUS_LENGTH


def test_attention_many_requests():
    """More requests than a CTA has threads, lengths from 0 to a few pages."""
    rng = np.random.default_rng(11)
    lengths = rng.integers(0, 200, 300).tolist()
    check_attention(rand_q(rng, 300, 1, 4, 64, "bf16"), Cache(rng, lengths, 2, 16, 64, "bf16"))


@pytest.mark.parametrize("R,W,H_q,H_kv,d,dtype", [(700, 1, 4, 2, 64, "bf16"), (33, 20, 4, 4, 64, "bf16"),
                                                  (500, 5, 8, 2, 128, "bf16"), (100, 1, 3, 1, 40, "f32")])
def test_attention_batches_longer_than_a_warp(R, W, H_q, H_kv, d, dtype):
    rng = np.random.default_rng(R)
    lengths = rng.integers(0, 40, R)
    lengths[R // 2] = 700
    cache = Cache(rng, lengths.tolist(), H_kv, 16, d, dtype, row_pages=45)
    check_attention(rand_q(rng, R, W, H_q, d, dtype), cache, dtype=dtype)


def test_attention_output_on_any_boundary():
    """o, q and the pools at addresses that rule the vector paths out."""
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(15)

    def shifted(t):
        u = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
        return u.copy_(t)

    for W, lengths in ((1, [40, 7]), (1, [600, 7]), (24, [300, 0])):
        cache = Cache(rng, lengths, 2, 16, 128, "bf16")
        q = rand_q(rng, 2, W, 8, 128, "bf16")
        k, v, table, n = cache.dev()
        ref = L.onela_paged_attention(q, k, v, table, n)
        got = [L.onela_paged_attention(q, k, v, table, n, out=shifted(q)),
               L.onela_paged_attention(shifted(q), shifted(k), shifted(v), table, n)]
        check_attention(q, cache)
        # Two kernels' results: each off by at most 2^-8 of its row's sum p |v|
        # (P's rounding; that sum is at most max |v|) and half a step of o;
        # the fp32 sums' part (below 2^-12) fits in the 1 % on top.
        vmax = cache.v[torch.isfinite(cache.v)].abs().max().double()
        for o in got:
            assert ((o.double() - ref.double()).abs() <= 1.01 * 2.0 ** -7 * (ref.double().abs() + vmax)).all()


def test_attention_long_row_is_split():
    """A row long enough for many pieces, against torch in 64 bits on the device."""
    import linear_attention_beam_shared_b200 as L
    torch.manual_seed(0)
    n, page, H, d = 70001, 64, 2, 128
    pages = n // page + 1
    for W, kernel in ((1, 0), (1, 1), (24, 0)):
        k, v = (torch.randn(pages, H, page, d, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        q = torch.randn(1, W, 8, d, device="cuda", dtype=torch.bfloat16)
        table = torch.randperm(pages, device="cuda").to(torch.int32)[None]
        o = L.onela_paged_attention(q, k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"), kernel=kernel)
        kk, vv = (x[table[0].long()].transpose(0, 1).reshape(H, -1, d)[:, :n].double() for x in (k, v))
        s = torch.einsum("whgd,hnd->whgn", q[0].double().reshape(W, H, 4, d), kk) * d ** -0.5
        p = torch.softmax(s, -1)
        ref = torch.einsum("whgn,hnd->whgd", p, vv).reshape(W, 8, d)
        spread = torch.einsum("whgn,hnd->whgd", p, vv.abs()).reshape(W, 8, d)
        # Weights: 2^-8 for bf16, and sums in pieces of at most 70001 terms:
        # n u = 0.0084 at worst; the scores' part is below 1e-4.
        lim = spread * (2.0 ** -8 + 2 * n * U + 1e-4) + 2.0 ** -8 * ref.abs()
        assert ((o[0].double() - ref).abs() <= lim).all()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements, its last pages in use."""
    import linear_attention_beam_shared_b200 as L
    H, page, d = 8, 64, 128
    pages = 2 ** 31 // (H * page * d) + 40
    k = torch.zeros((pages, H, page, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    torch.manual_seed(1)
    for W in (1, 20):
        kn, vn = (torch.randn(1, 200, H, d, device="cuda").bfloat16() for _ in range(2))
        table = torch.arange(pages - 4, pages, device="cuda", dtype=torch.int32)[None]
        L.onela_cache_write(kn, vn, k, v, table, torch.zeros(1, dtype=torch.int32, device="cuda"))
        q = torch.randn(1, W, 8, d, device="cuda").bfloat16()
        n = torch.tensor([200], dtype=torch.int32, device="cuda")
        small = (k[-4:].clone(), v[-4:].clone(), torch.arange(4, device="cuda", dtype=torch.int32)[None])
        assert torch.equal(small[0][0, :, 5], kn[0, 5])
        assert torch.equal(L.onela_paged_attention(q, k, v, table, n), L.onela_paged_attention(q, *small, n))
        m = torch.rand((1, H, 256), device="cuda")
        out = [torch.zeros_like(small[0][:2]), torch.zeros_like(small[0][:2]), torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"),
               torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(1, H, 128, device="cuda")]
        out2 = [t.clone() for t in out]
        L.onela_cache_evict(k, v, table, n, m, 100, 7, *out)
        L.onela_cache_evict(*small, n, m, 100, 7, *out2)
        assert all(torch.equal(a, b) for a, b in zip(out, out2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n,H,d,page,spaced", [
    (1, 1, 1, 1, 1, False), (3, 40, 2, 64, 16, False), (2, 33, 3, 37, 5, False), (70, 1, 4, 128, 1, True),
    (2, 19, 2, 6, 8, True)])
def test_cache_write(B, n, H, d, page, spaced, dtype):
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(B + n + d)
    start = rng.integers(0, 9, B).astype(np.int32)
    row_pages = -(-(n + 9) // page)
    pages = B * row_pages + 2
    table = rng.permutation(pages)[:B * row_pages].reshape(B, row_pages).astype(np.int32)
    counts = rng.integers(0, n + 1, B).astype(np.int32)
    pools = [torch.from_numpy(rng.standard_normal((pages, H, page, d)).astype(np.float32)).to(DT[dtype]).cuda() for _ in range(2)]
    if spaced:
        wide = rand_q(rng, B, n, 2 * H + 1, d, dtype)
        k, v = wide[:, :, :H], wide[:, :, H:2 * H]
    else:
        k, v = rand_q(rng, B, n, H, d, dtype), rand_q(rng, B, n, H, d, dtype)
    for c in (None, counts):
        kp, vp = pools[0].clone(), pools[1].clone()
        L.onela_cache_write(k, v, kp, vp, torch.from_numpy(table).cuda(), torch.from_numpy(start).cuda(),
                            counts=None if c is None else torch.from_numpy(c).cuda())
        np.testing.assert_array_equal(f64(kp), layers.cache_write(f64(k), f64(pools[0]), table, start, c))
        np.testing.assert_array_equal(f64(vp), layers.cache_write(f64(v), f64(pools[1]), table, start, c))


def test_cache_write_drops_what_does_not_fit():
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(0)
    k, v = rand_q(rng, 4, 6, 2, 64, "bf16"), rand_q(rng, 4, 6, 2, 64, "bf16")
    pool = rand_q(rng, 5, 2, 4, 64, "bf16")
    table = np.array([[0, 1], [2, 9], [-1, 3], [4, 4]], np.int32)
    start, counts = np.array([5, 0, 0, -2], np.int32), np.array([6, 6, 9, 4], np.int32)
    for c, want in ((None, 3), (counts, 3)):
        kp, vp = pool.clone(), pool.clone()
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        L.onela_cache_write(k, v, kp, vp, torch.from_numpy(table).cuda(), torch.from_numpy(start).cuda(),
                            counts=None if c is None else torch.from_numpy(c).cuda(), status=st)
        np.testing.assert_array_equal(f64(kp), layers.cache_write(f64(k), f64(pool), table, start, c))
        assert st.item() == want


def run_evict(cache, mass, keep, recent, H, page, d, dtype, kept=True, bad_dst=False, status=None):
    import linear_attention_beam_shared_b200 as L
    R = len(cache.lengths)
    rng = np.random.default_rng(5)
    dr = -(-keep // page) + 1
    pages = R * dr + 2
    dt = rng.permutation(pages)[:R * dr].reshape(R, dr).astype(np.int32)
    if bad_dst:
        dt[0, 0] = pages
    dk, dv = (torch.full((pages, H, page, d), 5.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    dm = torch.full((R, H, dr * page), -2.0, device="cuda")
    dl = torch.full((R,), -9, dtype=torch.int32, device="cuda")
    kp = torch.full((R, H, keep), -7, dtype=torch.int32, device="cuda") if kept else None
    ref = layers.cache_evict(f64(cache.k), f64(cache.v), cache.table, cache.lengths, mass, keep, recent, f64(dk), f64(dv), dt, f64(dm))
    k, v, table, lengths = cache.dev()
    L.onela_cache_evict(k, v, table, lengths, torch.from_numpy(mass).cuda(), keep, recent, dk, dv,
                        torch.from_numpy(dt).cuda(), dl, dm, kept=kp, status=status)
    got = [f64(dk), f64(dv), f64(dm), dl.cpu().numpy(), kp.cpu().numpy() if kept else ref[4]]
    for a, b, name in zip(got, ref, ("k", "v", "mass", "lengths", "kept")):
        np.testing.assert_array_equal(a, b, err_msg=name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lengths,H,page,d,keep,recent", [
    ([1], 1, 16, 64, 1, 0), ([10, 0, 200], 2, 16, 64, 30, 8), ([500, 30], 3, 8, 37, 64, 64), ([2100], 2, 64, 128, 1000, 1),
    ([64, 65], 1, 1, 6, 64, 0), ([5000], 1, 32, 128, 4000, 100), ([33], 2, 4, 5, 40, 7)])
@pytest.mark.parametrize("kind", ["smooth", "ties", "specials"])
def test_evict_matches_oracle(lengths, H, page, d, keep, recent, kind, dtype):
    rng = np.random.default_rng(len(lengths) + keep)
    cache = Cache(rng, lengths, H, page, d, dtype)
    shape = (len(lengths), H, cache.row_pages * page)
    m = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        m = rng.integers(0, 4, shape).astype(np.float32)
    if kind == "specials":
        pick = rng.random(shape)
        m[pick < 0.3] = 0.0
        m[pick < 0.15] = -0.0
        m[pick < 0.1] = np.nan
        m[pick < 0.05] = np.inf
        m[pick < 0.02] = -np.inf
        m[pick < 0.01] = -1.5
    run_evict(cache, m, keep, recent, H, page, d, dtype)


def test_evict_all_weights_equal_and_long_rows():
    rng = np.random.default_rng(2)
    cache = Cache(rng, [9000, 40000], 1, 64, 8, "bf16")
    shape = (2, 1, cache.row_pages * 64)
    run_evict(cache, np.ones(shape, np.float32), 3000, 5, 1, 64, 8, "bf16")
    run_evict(cache, np.full(shape, np.nan, np.float32), 3000, 0, 1, 64, 8, "bf16", kept=False)
    run_evict(cache, rng.random(shape).astype(np.float32), 39999, 0, 1, 64, 8, "bf16")


@pytest.mark.parametrize("kind", ["smooth", "nan", "few_numbers", "levels"])
@pytest.mark.parametrize("n,keep", [(16384, 9000), (16385, 16000), (40000, 25000), (131072, 100000), (131073, 60000),
                                    (150000, 149000)])
def test_evict_rows_of_several_ctas(n, keep, kind):
    """Rows up to and past what a cluster keeps in shared memory, with ties
    that run across its CTAs' borders."""
    rng = np.random.default_rng(n)
    cache = Cache(rng, [n, n // 3], 1, 64, 4, "f32")
    shape = (2, 1, cache.row_pages * 64)
    m = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "nan":
        m[:] = np.nan
    if kind == "few_numbers":
        m = np.where(rng.random(shape) < 0.9, np.float32(np.nan), m)
    if kind == "levels":
        m = (1 + rng.integers(0, 3, shape) * 2.0 ** -20).astype(np.float32)
    run_evict(cache, m, keep, 7, 1, 64, 4, "f32")


def test_evict_bad_pages_and_lengths():
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(4)
    cache = Cache(rng, [100, 64], 2, 16, 64, "bf16", row_pages=8)
    cache.table[0, 3] = -2
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m = rng.random((2, 2, 128)).astype(np.float32)
    run_evict(cache, m, 70, 10, 2, 16, 64, "bf16", bad_dst=True, status=st)
    assert st.item() == L.ONELA_STATUS_PAGE
    cache.lengths[:] = (-3, 1000)
    cache.table[1, 6] = 10 ** 9
    st.zero_()
    run_evict(cache, m, 70, 10, 2, 16, 64, "bf16", status=st)
    assert st.item() == L.ONELA_STATUS_PAGE | L.ONELA_STATUS_LENGTH


NORMS = [(1, 64, 64), (5, 256, 64), (3, 2048, 2048), (2, 1000, 1000), (4, 37, 37), (3, 60, 20), (2, 8192, 8192),
         (2, 4104, 4104), (2, 1536, 96), (1, 16384, 128), (1, 32768, 32768), (2, 5000, 8), (3, 48, 2), (700, 128, 128), (1, 32768, 1), (2, 30000, 3), (3, 31, 1), (1, 1, 1)]


@pytest.mark.parametrize("parts", ["all", "heads", "post", "pre", "residual"])
@pytest.mark.parametrize("ydt,dtype", [("f32", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")])
@pytest.mark.parametrize("N,D,group", NORMS)
def test_block_norm_matches_oracle(N, D, group, ydt, dtype, parts):
    """Error of x': u is a product of y, rsqrt of a D-term mean, w, act, alpha,
    scale, each rounded (and the mean off by D u / 2 relative in the rsqrt):
    |u| (D u + 16 u), plus the additions and half a step of the output; n' adds
    D u + 16 u again relative to n, and x' enters it through w / rms with its own error."""
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(N + D)
    pick = dict(all="yxgwsp", heads="ygw", post="yxw", pre="xp", residual="yxgsp")[parts]
    t = lambda dt: torch.from_numpy(rng.standard_normal((N, D)).astype(np.float32)).to(DT[dt]).cuda()  # noqa: E731
    vec = lambda n: torch.from_numpy((1 + 0.2 * rng.standard_normal(n)).astype(np.float32)).cuda()     # noqa: E731
    a = dict(y=t(ydt) if "y" in pick else None, x=t(dtype) if "x" in pick else None,
             gate=t(dtype) * 3 if "g" in pick else None, w_post=vec(group) if "w" in pick else None,
             scale=vec(D) if "s" in pick else None, w_pre=vec(D) if "p" in pick else None)
    act = "none" if a["gate"] is None else ("silu" if D % 3 else "sigmoid")
    x, n = L.onela_block_norm(**a, gate_act=act, alpha=0.75, dtype=dtype)
    host = {k: None if v is None else f64(v) for k, v in a.items()}
    rx, rn = layers.block_norm(**host, act=act, alpha=0.75)
    u = np.abs(rx - (host["x"] if a["x"] is not None else 0)) if a["y"] is not None else np.zeros_like(rx)
    ex = u * (D + 16) * U + np.abs(rx) * 2 * U
    assert (np.abs(f64(x) - rx) <= ex + HALF[dtype] * np.abs(rx) * 1.01 + 1e-37).all()
    assert (n is None) == (rn is None)
    if n is not None:
        factor = np.abs(host["w_pre"]) / np.sqrt((rx ** 2).mean(1, keepdims=True) + 1e-6)
        lim = ex * factor + np.abs(rn) * ((D + 16) * U + ex.max() / np.sqrt((rx ** 2).mean())) + HALF[dtype] * np.abs(rn) * 1.01
        assert (np.abs(f64(n) - rn) <= lim).all()


def test_block_norm_strides_in_place_and_parts():
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(1)
    wide = torch.from_numpy(rng.standard_normal((6, 400)).astype(np.float32)).cuda()
    w = torch.ones(128, device="cuda")
    for lo in (0, 3, 8):
        y, g, x = wide[:, lo:lo + 128], wide[:, 130 + lo:258 + lo], wide[:, 260 + lo:388 + lo]
        a = L.onela_block_norm(y, x=x, gate=g, gate_act="silu", w_post=w, w_pre=w)
        b = L.onela_block_norm(y.contiguous(), x=x.contiguous(), gate=g.contiguous(), gate_act="silu", w_post=w, w_pre=w)
        for s, t in zip(a, b):
            # The same sums in another order: both within (D + 16) u of the row's scale.
            assert ((s - t).abs() <= 2 * (128 + 16) * U * t.abs().max()).all()
        xd = x.contiguous()
        L.onela_block_norm(y.contiguous(), x=xd, gate=g.contiguous(), gate_act="silu", w_post=w, w_pre=w, x_out=xd)
        assert torch.equal(xd, b[0])
        none, n = L.onela_block_norm(y.contiguous(), x=x.contiguous(), gate=g.contiguous(), gate_act="silu", w_post=w, w_pre=w, want_x=False)
        assert none is None and torch.equal(n, b[1])
    x, n = L.onela_block_norm(torch.zeros((0, 8), device="cuda"), w_pre=torch.ones(8, device="cuda"))
    assert x.shape == n.shape == (0, 8)
    z, n = L.onela_block_norm(torch.zeros((2, 64), device="cuda"), w_post=torch.ones(64, device="cuda"), w_pre=torch.ones(64, device="cuda"))
    assert (z == 0).all() and (n == 0).all()


def test_capture_before_any_call():
    """In a process of its own: the first calls ever are captured, then replayed."""
    import subprocess
    import sys
    code = """
import torch, linear_attention_beam_shared_b200 as L
i32 = dict(dtype=torch.int32, device="cuda")
k, v = (torch.randn(40, 2, 16, 64, device="cuda").bfloat16() for _ in range(2))
table, n = torch.arange(32, **i32)[None], torch.full((1,), 500, **i32)
mass = torch.zeros(1, 2, 512, device="cuda")
dst = (torch.zeros_like(k), torch.zeros_like(v), torch.arange(8, **i32)[None], torch.zeros(1, **i32), torch.zeros(1, 2, 128, device="cuda"))
x = torch.randn(4, 256, device="cuda").bfloat16()
w = torch.ones(256, device="cuda")
new = torch.randn(1, 1, 2, 64, device="cuda").bfloat16()
qs = [torch.randn(1, W, 8, 64, device="cuda").bfloat16() for W in (1, 20)] + [torch.randn(1, 2, 8, 64, device="cuda")]
kf, vf = k.float(), v.float()
start = torch.full((1,), 500, **i32)
def run():
    L.onela_cache_write(new, new, k, v, table, start)
    o = [L.onela_paged_attention(q, *((k, v) if q.dtype == torch.bfloat16 else (kf, vf)), table, n, mass_out=mass) for q in qs]
    L.onela_cache_evict(k, v, table, n, mass, 100, 9, *dst)
    return o + list(L.onela_block_norm(x, x=x, w_post=w, w_pre=w))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = run()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in out] + [t.clone() for t in dst]
ref = run() + list(dst)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, ref))
raw = L.onela_paged_attention(qs[0], k, v, table, n, stream=0)
torch.cuda.synchronize()
assert torch.equal(raw, L.onela_paged_attention(qs[0], k, v, table, n))
print("ok")
"""
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stderr[-2000:]


@pytest.mark.parametrize("how", ["graph", "stream", "raw"])
def test_graph_capture_and_other_streams(how):
    """All four in one captured graph, replayed on new inputs; or on a stream
    that is not the current one.  Bitwise the same as plain calls."""
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(12)
    R, W, H_q, H, d, page = 2, 20, 8, 2, 64, 16
    cache = Cache(rng, [300, 90], H, page, d, "bf16")
    k, v, table, lengths = cache.dev()
    q = rand_q(rng, R, W, H_q, d, "bf16")
    bk, bv, bt, bl = draw_beam(rng, R, W, H, d, "bf16", np.full((R, W), 3))
    bt = torch.arange(R * W * 3, dtype=torch.int32).reshape(R, W, 3).cuda()
    bk, bv = torch.zeros(R * W * 3, H, 1, d, device="cuda").bfloat16(), torch.zeros(R * W * 3, H, 1, d, device="cuda").bfloat16()
    bl = torch.full((R, W), 3, dtype=torch.int32, device="cuda")
    kn = rand_q(rng, R * W, 3, H, d, "bf16")
    start = torch.zeros(R * W, dtype=torch.int32, device="cuda")
    mass = torch.zeros(R, H, cache.row_pages * page, device="cuda")
    dst = [torch.zeros(R * 4, H, page, d, device="cuda").bfloat16() for _ in range(2)]
    dt = torch.arange(R * 4, dtype=torch.int32, device="cuda").reshape(R, 4)
    dl, dm = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(R, H, 64, device="cuda")
    w = torch.ones(H_q * d, device="cuda")
    sizes = (R, W, H_q, H, d, "bf16", page, k.shape[0], table.shape[1], 1, bk.shape[0], 3)
    scratch = torch.empty(L.onela_paged_attention_scratch_bytes(*sizes, want_mass=True), dtype=torch.uint8, device="cuda")

    def run(stream=None, scratch=None):
        L.onela_cache_write(kn, kn, bk, bv, bt.reshape(R * W, 3), start, stream=stream)
        o = L.onela_paged_attention(q, k, v, table, lengths, beam=(bk, bv, bt, bl), mass_out=mass, scratch=scratch, stream=stream)
        L.onela_cache_evict(k, v, table, lengths, mass, 60, 10, *dst, dt, dl, dm, stream=stream)
        x, n = L.onela_block_norm(o.reshape(R * W, H_q * d), x=q.reshape(R * W, H_q * d), w_post=w, w_pre=w, stream=stream)
        return o, x, n

    def snap(out):
        torch.cuda.synchronize()
        return [t.clone() for t in (*out, *dst, dl, dm, mass[:, :, :90])]

    run()
    torch.cuda.synchronize()
    if how == "graph":
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(scratch=scratch)
        for i in range(2):
            q.copy_(rand_q(rng, R, W, H_q, d, "bf16"))
            g.replay()
            got = snap(out)
            assert all(torch.equal(a, b) for a, b in zip(got, snap(run())))
    else:
        s = torch.cuda.Stream()
        q.copy_(rand_q(rng, R, W, H_q, d, "bf16"))
        torch.cuda.synchronize()
        got = snap(run(stream=s if how == "stream" else s.cuda_stream))
        assert all(torch.equal(a, b) for a, b in zip(got, snap(run())))


@pytest.mark.parametrize("W", [1, 40])
def test_attention_is_deterministic(W):
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(13)
    cache = Cache(rng, [3000, 10, 999], 2, 16, 128, "bf16")
    q = rand_q(rng, 3, W, 8, 128, "bf16")
    k, v, table, lengths = cache.dev()
    m = torch.zeros(3, 2, cache.row_pages * 16, device="cuda")
    a = L.onela_paged_attention(q, k, v, table, lengths, mass_out=m)
    m1 = m.clone()
    for _ in range(5):
        assert torch.equal(a, L.onela_paged_attention(q, k, v, table, lengths, mass_out=m))
        assert torch.equal(m, m1)


def test_hybrid_decode():
    """The operators as a hybrid decoder's beam search runs them, three steps:
    per-head gated norm of the GDN step's o, residual and pre-norm, then full
    attention over the prompt's pages and the beams' own tokens, whose table is
    the GDN handle's ancestry; the weights added up over the steps, and the
    prompt's cache cut by them at the end.  Each operator against the oracle on the inputs it was
    given."""
    import linear_attention_beam_shared_b200 as L
    import synth
    wl = synth.workload("tiny").replace(qkv_dtype="bf16", d_k=64, d_v=64)
    R, H, d, W, T = wl.R, wl.H, 64, wl.W, wl.T
    S0 = synth.cast_state(synth.draw_s0_direct(wl), "f32")
    steps = synth.draw_decode(wl)
    rng = np.random.default_rng(14)
    dec = L.BeamDecoder(R, H, d, d, W, T, "f32", "bf16")
    page, n0 = 16, 100
    cache = Cache(rng, [n0] * R, H, page, d, "bf16")
    k, v, table, lengths = cache.dev()
    slots = T * R * W
    bk = torch.zeros((slots, H, 1, d), dtype=torch.bfloat16, device="cuda")
    bv = torch.zeros_like(bk)
    mass = torch.zeros((R, H, cache.row_pages * page), device="cuda")
    total = np.zeros(mass.shape)
    w_head, w_all = torch.ones(d, device="cuda"), torch.ones(H * d, device="cuda")
    resid = None
    base = torch.arange(R * W, dtype=torch.int32, device="cuda").reshape(R, W)
    try:
        dec.set_prompt_state(S0.cuda())
        for t, s in enumerate(steps, start=1):
            g = {n: (x.cuda() if isinstance(x, torch.Tensor) else x) for n, x in s.items()}
            o = dec.step(g["q"], g["k"], g["v"], g["g"], g["beta"], g["parents"])
            gate = rand_q(rng, R * W, H, 1, d, "bf16").reshape(-1, d)
            heads, _ = L.onela_block_norm(o.reshape(-1, d), gate=gate, gate_act="silu", w_post=w_head, dtype="bf16")
            want, _ = layers.block_norm(y=f64(o).reshape(-1, d), gate=f64(gate), act="silu", w_post=np.ones(d))
            assert (np.abs(f64(heads) - want) <= np.abs(want) * (2.0 ** -8 + 100 * U)).all()
            x, nrm = L.onela_block_norm(heads.reshape(R * W, H * d), x=resid, w_pre=w_all)
            resid = x
            q = nrm.reshape(R, W, H, d)
            kn, vn = rand_q(rng, R * W, 1, H, d, "bf16"), rand_q(rng, R * W, 1, H, d, "bf16")
            new = base.reshape(-1, 1) + (t - 1) * R * W
            L.onela_cache_write(kn, vn, bk, bv, new, torch.zeros(R * W, dtype=torch.int32, device="cuda"))
            # The ancestors' slots level by level, then the beam's own.
            anc = dec.ancestry(t)
            first = (torch.arange(R, device="cuda", dtype=torch.int32) * W)[:, None, None]
            level = torch.arange(t - 1, device="cuda", dtype=torch.int32)[None, None] * (R * W)
            btab = torch.cat([anc + first + level, new.reshape(R, W, 1)], -1).contiguous()
            blen = torch.full((R, W), t, dtype=torch.int32, device="cuda")
            beam = (bk, bv, btab.cpu().numpy(), blen.cpu().numpy())
            got = check_attention(q.contiguous(), cache, beam=beam)
            o2 = L.onela_paged_attention(q, k, v, table, lengths, beam=(bk, bv, btab, blen), mass=mass, mass_out=mass)
            assert torch.equal(got, o2)
            _, _, m, _ = layers.paged_attention(f64(q), *cache.host(), beam=(f64(bk), f64(bv), beam[2], beam[3]))
            total += m
            y, _ = L.onela_block_norm(o2.reshape(R * W, H * d), x=resid, w_post=w_all, scale=w_all)
            assert torch.isfinite(y).all()
        assert dec.status() == 0
        assert np.abs(f64(mass) - total)[:, :, :n0].max() <= total.max() * 1e-4
        run_evict(cache, mass.cpu().numpy(), 40, 8, H, page, d, "bf16")
    finally:
        dec.close()


def test_evict_within_one_pool_and_attend_again():
    """The destination pages may lie in the source's pool; the cut cache is
    then read like any other, and what was not moved is untouched."""
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(20)
    R, H, page, d, keep = 2, 2, 16, 128, 40
    cache = Cache(rng, [150, 30], H, page, d, "bf16", row_pages=11, spare=10)
    k, v, table, lengths = cache.dev()
    free = np.setdiff1d(np.arange(k.shape[0]), cache.table).astype(np.int32)
    new = torch.from_numpy(free[:R * 3].reshape(R, 3)).cuda()
    mass = rng.random((R, H, 11 * page)).astype(np.float32)
    before_k, before_v = f64(k), f64(v)
    dl, dm = torch.zeros(R, dtype=torch.int32, device="cuda"), torch.zeros(R, H, 48, device="cuda")
    L.onela_cache_evict(k, v, table, lengths, torch.from_numpy(mass).cuda(), keep, 5, k, v, new, dl, dm)
    rk, rv, rm, rn, kept = layers.cache_evict(before_k, before_v, cache.table, cache.lengths, mass, keep, 5, before_k,
                                              before_v, new.cpu().numpy(), np.zeros((R, H, 48)))
    np.testing.assert_array_equal(f64(k), rk)
    np.testing.assert_array_equal(f64(v), rv)
    np.testing.assert_array_equal(dl.cpu().numpy(), rn)
    cut = Cache.__new__(Cache)
    cut.k, cut.v, cut.table, cut.lengths, cut.row_pages = k, v, new.cpu().numpy(), rn, 3
    check_attention(rand_q(rng, R, 1, 4, d, "bf16"), cut)
    # Per head: the same as attention over the kept tokens of the old cache.
    assert (kept[0, 0] != kept[0, 1]).any()


def test_two_streams_and_two_graphs_at_once():
    """Calls of their own scratch on two streams, and two captured graphs
    replayed at once, give what they give alone."""
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(21)
    jobs = []
    for W in (1, 40):
        cache = Cache(rng, [3000, 700], 2, 16, 128, "bf16")
        k, v, table, lengths = cache.dev()
        q = rand_q(rng, 2, W, 8, 128, "bf16")
        m = torch.zeros(2, 2, cache.row_pages * 16, device="cuda")
        jobs.append((q, k, v, table, lengths, m))

    def call(j, s=None):
        q, k, v, table, lengths, m = j
        return L.onela_paged_attention(q, k, v, table, lengths, mass_out=m, stream=s)

    ref = [(call(j).clone(), j[5].clone()) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [[] for _ in jobs]
    for _ in range(5):
        for i, (j, s) in enumerate(zip(jobs, streams)):
            outs[i].append(call(j, s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, ref[i][0]) for o in outs[i]) and torch.equal(jobs[i][5], ref[i][1])
    graphs = []
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = call(j)
        graphs.append((g, o))
    for _ in range(5):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(graphs[i][1], ref[i][0]) and torch.equal(jobs[i][5], ref[i][1])


@pytest.mark.parametrize("G,W", [(1, 40), (3, 20), (64, 1), (96, 1), (32, 5), (5, 60)])
def test_attention_group_sizes(G, W):
    """Grouped heads that do and do not divide a box of 64 query rows."""
    rng = np.random.default_rng(G)
    blen = rng.integers(0, 4, (2, W))
    blen[0, 0] = 3
    cache = Cache(rng, [130, 64], 2, 16, 64, "bf16")
    check_attention(rand_q(rng, 2, W, 2 * G, 64, "bf16"), cache, beam=draw_beam(rng, 2, W, 2, 64, "bf16", blen),
                    mass=rng.random((2, 2, cache.row_pages * 16)).astype(np.float32))


@pytest.mark.parametrize("dtype,d,W", [("bf16", 64, 1), ("bf16", 64, 30), ("f32", 64, 1), ("bf16", 37, 2)])
def test_attention_nan_is_not_hidden(dtype, d, W):
    """A NaN query gives NaN rows and weights, over a prompt, beam tokens alone, or both."""
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(23)
    for lengths, blen in (([300], 0), ([0], 3), ([20], 0), ([300], 3)):
        cache = Cache(rng, lengths, 2, 16, d, dtype, row_pages=20)
        q = rand_q(rng, 1, W, 4, d, dtype)
        q[0, 0, 0, 0] = float("nan")
        k, v, table, n = cache.dev()
        beam = None
        if blen:
            b = draw_beam(rng, 1, W, 2, d, dtype, np.full((1, W), blen))
            beam = (b[0], b[1], torch.from_numpy(b[2]).cuda(), torch.from_numpy(b[3]).cuda())
        lse, m = torch.zeros(1, W, 4, device="cuda"), torch.zeros(1, 2, 320, device="cuda")
        o = L.onela_paged_attention(q, k, v, table, n, beam=beam, lse=lse, mass_out=m)
        assert torch.isnan(o[0, 0, 0].float()).all() and torch.isnan(lse[0, 0, 0])
        assert torch.isfinite(o[0, 0, 1:].float()).all() and torch.isfinite(o[0, 1:].float()).all()
        assert torch.isnan(m[0, 0, :lengths[0]]).all() and torch.isfinite(m[0, 1]).all()


def test_attention_other_requests_nan_stays_theirs():
    """NaN in one request's query and cache leaves the others' rows alone."""
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(22)
    for W in (1, 20, 70):
        cache = Cache(rng, [200, 90, 100], 2, 16, 64, "bf16")
        q = rand_q(rng, 3, W, 8, 64, "bf16")
        k, v, table, lengths = cache.dev()
        m = torch.zeros(3, 2, cache.row_pages * 16, device="cuda")
        ref = L.onela_paged_attention(q, k, v, table, lengths, mass_out=m).clone()
        rm = m.clone()
        q[1] = float("nan")
        k[table[1, 0].long()] = float("nan")
        o = L.onela_paged_attention(q, k, v, table, lengths, mass_out=m)
        assert torch.isnan(o[1].float()).all()
        for r in (0, 2):
            assert torch.equal(o[r], ref[r]) and torch.equal(m[r], rm[r])


@pytest.mark.parametrize("W", [1, 24])
def test_back_to_back_calls_see_each_other(W):
    """A chain of dependent calls launched without a wait, each kernel allowed
    to start while the one before it ends: bitwise what it gives with a device
    wait after every call."""
    import linear_attention_beam_shared_b200 as L
    R, H_q, H, d, page, n0, steps = 2, 8, 2, 64, 16, 90, 40
    i32 = dict(dtype=torch.int32, device="cuda")

    def run(wait):
        gen = torch.Generator(device="cuda").manual_seed(5)
        rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()   # noqa: E731
        k, v = rnd(R * 20 + 1, H, page, d), rnd(R * 20 + 1, H, page, d)
        tables = [torch.arange(R * 10, **i32).reshape(R, 10), torch.arange(R * 10, R * 20, **i32).reshape(R, 10)]
        lens = [torch.full((R,), n0, **i32), torch.zeros(R, **i32)]
        mass = [torch.zeros(R, H, 10 * page, device="cuda") for _ in range(2)]
        bk, bv = rnd(R * W, H, 1, d), rnd(R * W, H, 1, d)
        bt, bl = torch.arange(R * W, **i32).reshape(R, W, 1), torch.ones((R, W), **i32)
        x, w = rnd(R * W, H_q * d), 1 + 0.1 * rnd(H_q * d).float()
        sync = torch.cuda.synchronize if wait else (lambda: None)
        torch.cuda.synchronize()
        cur, outs = 0, []
        for t in range(steps):
            _, q = L.onela_block_norm(x=x, w_pre=w, want_x=False)
            sync()
            new = q.view(R * W, 1, H_q, d)
            L.onela_cache_write(new[:, :, :H], new[:, :, H:2 * H], bk, bv, bt.view(R * W, 1), torch.zeros(R * W, **i32))
            sync()
            L.onela_cache_write(new.view(R, W, H_q, d)[:, :1, :H], new.view(R, W, H_q, d)[:, :1, H:2 * H], k, v,
                                tables[cur], lens[cur])
            sync()
            lens[cur] += 1
            o = L.onela_paged_attention(q.view(R, W, H_q, d), k, v, tables[cur], lens[cur], beam=(bk, bv, bt, bl),
                                        mass=mass[cur], mass_out=mass[cur])
            sync()
            if t % 7 == 6:
                L.onela_cache_evict(k, v, tables[cur], lens[cur], mass[cur], 80, 8, k, v, tables[1 - cur], lens[1 - cur],
                                    mass[1 - cur])
                sync()
                mass[1 - cur][:, :, 80:] = 0
                mass[cur].zero_()
                cur = 1 - cur
            x, _ = L.onela_block_norm(o.view(R * W, H_q * d), x=x, w_post=w, alpha=0.5)
            sync()
            outs.append(x)
        torch.cuda.synchronize()
        return outs + [k, v, lens[cur], mass[cur]]

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)
        assert torch.isfinite(a.float()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D", [(2, 64), (3, 37), (2, 5000), (2400, 256)])
def test_block_norm_shut_gates(N, D, dtype):
    """Gates of the type's lowest value: silu and sigmoid of them are 0, whatever u is."""
    import linear_attention_beam_shared_b200 as L
    dt = DT[dtype]
    y = torch.full((N, D), 30.0, device="cuda", dtype=dt)
    y[:, ::2] = -70.0
    x = torch.full((N, D), 2.0, device="cuda", dtype=dt)
    gate = torch.full((N, D), torch.finfo(dt).min, device="cuda", dtype=dt)
    w = torch.full((D,), 5.0, device="cuda")
    for act in ("silu", "sigmoid"):
        for post in (None, w):
            got, _ = L.onela_block_norm(y, x=x, gate=gate, gate_act=act, w_post=post)
            assert torch.equal(got, x)


def test_capture_of_two_branches():
    """A captured graph whose streams part and meet: calls that follow copies,
    clears and one another across streams; bitwise the same as plain calls."""
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(77)
    R, W, H_q, H, d, page = 2, 3, 8, 2, 64, 16
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = Cache(rng, [300, 90], H, page, d, "bf16")
    k, v, table, lengths = cache.dev()
    q = rand_q(rng, R, W, H_q, d, "bf16")
    bk, bv = (torch.zeros(R * W, H, 1, d, device="cuda").bfloat16() for _ in range(2))
    bt, one, zero = torch.arange(R * W, **i32).reshape(R, W, 1), torch.ones(R, W, **i32), torch.zeros(R * W, **i32)
    new = rand_q(rng, R * W, 1, H, d, "bf16")
    into, mass = torch.zeros_like(new), torch.zeros(R, H, cache.row_pages * page, device="cuda")
    y, x = rand_q(rng, R * W, 1, 1, H_q * d, "bf16").reshape(R * W, -1), rand_q(rng, R * W, 1, 1, H_q * d, "bf16").reshape(R * W, -1)
    w = torch.ones(H_q * d, device="cuda")

    def run(main, side):
        side.wait_stream(main)
        with torch.cuda.stream(side):
            into.copy_(new)
            L.onela_cache_write(into, into, bk, bv, bt.reshape(R * W, 1), zero)
        mass.zero_()
        _, n = L.onela_block_norm(y, x=x, w_post=w, w_pre=w)
        main.wait_stream(side)  # the next call follows a kernel on either stream
        o = L.onela_paged_attention(q, k, v, table, lengths, beam=(bk, bv, bt, one), mass=mass, mass_out=mass)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            bk.zero_()  # after the attention has read it
        a, b = L.onela_block_norm(o.reshape(R * W, -1), x=n, w_post=w, w_pre=w)
        main.wait_stream(side)
        return o, n, a, b

    side = torch.cuda.Stream()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run(s, side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(torch.cuda.current_stream(), side)
    for i in range(3):
        new.copy_(rand_q(rng, R * W, 1, H, d, "bf16"))
        y.copy_(rand_q(rng, R * W, 1, 1, H_q * d, "bf16").reshape(R * W, -1))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, mass[:, :, :90])]
        with torch.cuda.stream(s):
            ref = run(s, side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (*ref, mass[:, :, :90])))
        assert (bk == 0).all()


def test_threads_on_streams_of_their_own():
    """Calls of all kinds from four host threads at once, bitwise as from one."""
    import threading
    import linear_attention_beam_shared_b200 as L
    rng = np.random.default_rng(78)
    i32 = dict(dtype=torch.int32, device="cuda")
    jobs = []
    for W in (1, 3, 20, 40):
        cache = Cache(rng, [500, 33], 2, 16, 64, "bf16")
        jobs.append((rand_q(rng, 2, W, 8, 64, "bf16"), cache.dev(), rand_q(rng, 2, 1, 2, 64, "bf16")))
    w = torch.ones(512, device="cuda")
    torch.cuda.synchronize()

    def run(i, into, stream):
        q, (k, v, table, lengths), new = jobs[i]
        with torch.cuda.stream(stream):
            mass = torch.zeros(2, 2, table.shape[1] * 16, device="cuda")
            kk, vv = k.clone(), v.clone()
            L.onela_cache_write(new, new, kk, vv, table, lengths - 1)
            o = L.onela_paged_attention(q, kk, vv, table, lengths, mass_out=mass)
            dst = [torch.zeros(8, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            n, m = torch.zeros(2, **i32), torch.zeros(2, 2, 64, device="cuda")
            L.onela_cache_evict(kk, vv, table, lengths, mass, 50, 7, *dst, torch.arange(8, **i32).reshape(2, 4), n, m)
            x, y = L.onela_block_norm(o.reshape(-1, 512), w_post=w, w_pre=w)
        stream.synchronize()
        into[i] = [o, mass, *dst, n, m, x, y]

    ref, errors = {}, []
    for i in range(4):
        run(i, ref, torch.cuda.current_stream())

    def many(i):
        try:
            stream, got = torch.cuda.Stream(), {}
            for _ in range(20):
                run(i, got, stream)
                if not all(torch.equal(a, b) for a, b in zip(got[i], ref[i])):
                    errors.append(f"job {i} differs")
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))

    threads = [threading.Thread(target=many, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
