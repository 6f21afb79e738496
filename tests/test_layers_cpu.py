"""Host-side refusals of the operators around a GDN layer, through the C ABI:
every check comes before the device is touched, so the pointers given here are
never used."""
import ctypes

import pytest

P = 4096  # an aligned address; never dereferenced


def attention(L, **change):
    f = dict(R=2, W=3, H_q=8, H_kv=2, d=64, dtype=1, kernel=0, page=16, pages=10, row_pages=40, beam_page=0,
             beam_pages=0, beam_row_pages=0, device=0, q_stride=8 * 64, scale=0.125)
    f.update(change)
    return L._layers.onela_attention_config(*[f[n] for n, _ in L._layers.onela_attention_config._fields_])


def call_attention(L, cfg, scratch_bytes=1 << 40, **change):
    a = dict(q=3 * P, k=P, v=P, table=P, lengths=P, bk=None, bv=None, bt=None, bl=None, mass=None, mass_out=None, o=P,
             lse=None, scratch=P)
    a.update(change)
    return L._lib.lib.onela_paged_attention(ctypes.addressof(cfg), *a.values(), scratch_bytes, None, None)


@pytest.mark.parametrize("field,value", [
    ("R", 0), ("R", 65536), ("W", 0), ("H_q", 0), ("H_q", 7), ("H_kv", 0), ("d", 0), ("d", 257), ("dtype", 2),
    ("kernel", 3), ("page", 0), ("pages", 0), ("row_pages", 0), ("row_pages", 1 << 27), ("beam_page", 1),
    ("device", -1), ("q_stride", 511), ("scale", 0.0), ("scale", float("nan")), ("scale", float("inf")), ("W", 16385),
    ("pages", 1 << 30)])
def test_attention_refuses_bad_config(field, value):
    import linear_attention_beam_shared_b200 as L
    cfg = attention(L, **{field: value})
    assert call_attention(L, cfg) == L.ONELA_ERR_ARG
    assert L._lib.lib.onela_paged_attention_scratch_bytes(ctypes.addressof(cfg), 0) == 0


@pytest.mark.parametrize("change", [
    dict(q=None), dict(k=None), dict(v=None), dict(table=None), dict(lengths=None), dict(o=None), dict(scratch=None),
    dict(scratch=P + 16), dict(q=P + 1), dict(lengths=P + 2), dict(o=P + 1), dict(mass=P), dict(bk=P), dict(bk=P, bv=P, bt=P, bl=P),
    dict(q=2 * P, o=2 * P)])
def test_attention_refuses_bad_pointers(change):
    import linear_attention_beam_shared_b200 as L
    assert call_attention(L, attention(L), **change) == L.ONELA_ERR_ARG


def test_attention_refuses_missing_beam_pointers_and_small_scratch():
    import linear_attention_beam_shared_b200 as L
    cfg = attention(L, beam_page=1, beam_pages=9, beam_row_pages=5)
    assert call_attention(L, cfg, bk=P, bv=P, bt=P) == L.ONELA_ERR_ARG
    need = L._lib.lib.onela_paged_attention_scratch_bytes(ctypes.addressof(cfg), 0)
    assert need > 0
    assert L._lib.lib.onela_paged_attention_scratch_bytes(ctypes.addressof(cfg), 1) > need
    # Scores are kept only where the kernel that runs needs them.
    wide, general = (attention(L, W=200, kernel=n) for n in (0, L.ONELA_KERNEL_SIMT))
    rows = 2 * 200 * 8
    sizes = [L._lib.lib.onela_paged_attention_scratch_bytes(ctypes.addressof(c), 1) for c in (wide, general)]
    assert sizes[1] > rows * 640 * 4 > sizes[0] - 40 * rows * 64 * 4
    # On pointers that rule the tensor cores out, the smaller scratch is refused.
    assert call_attention(L, wide, sizes[0], q=3 * P + 2, mass_out=P) == L.ONELA_ERR_SCRATCH
    assert call_attention(L, cfg, need - 1, bk=P, bv=P, bt=P, bl=P) == L.ONELA_ERR_SCRATCH
    assert L._lib.lib.onela_paged_attention(None, *[None] * 14, 0, None, None) == L.ONELA_ERR_ARG


@pytest.mark.parametrize("change", [dict(dtype=0, d=64), dict(d=80, q_stride=8 * 80)])
def test_attention_refuses_a_forced_kernel_it_cannot_run(change):
    import linear_attention_beam_shared_b200 as L
    assert call_attention(L, attention(L, kernel=L.ONELA_KERNEL_TC, **change)) == L.ONELA_ERR_UNSUPPORTED


def write_cfg(L, **change):
    f = dict(B=2, n=5, H_kv=2, d=64, dtype=1, page=16, pages=10, row_pages=4, device=0, k_stride=128, v_stride=128)
    f.update(change)
    return L._layers.onela_cache_write_config(*[f[n] for n, _ in L._layers.onela_cache_write_config._fields_])


@pytest.mark.parametrize("field,value", [
    ("B", 0), ("n", 0), ("H_kv", 0), ("d", 0), ("d", 300), ("dtype", -1), ("page", 0), ("pages", 0), ("row_pages", 0),
    ("device", -1), ("k_stride", 127), ("v_stride", 0), ("n", 1 << 30)])
def test_write_refuses_bad_config(field, value):
    import linear_attention_beam_shared_b200 as L
    cfg = write_cfg(L, **{field: value})
    assert L._lib.lib.onela_cache_write(ctypes.addressof(cfg), P, P, P, 2 * P, P, P, None, None, None) == L.ONELA_ERR_ARG


def test_write_refuses_bad_pointers():
    import linear_attention_beam_shared_b200 as L
    cfg = write_cfg(L)
    good = [P, P, P, 2 * P, P, P]
    for i in range(6):
        for bad in (None, P + 1):
            a = list(good)
            a[i] = bad
            assert L._lib.lib.onela_cache_write(ctypes.addressof(cfg), *a, None, None, None) == L.ONELA_ERR_ARG
    assert L._lib.lib.onela_cache_write(None, *good, None, None, None) == L.ONELA_ERR_ARG
    assert L._lib.lib.onela_cache_write(ctypes.addressof(cfg), *[P] * 6, None, None, None) == L.ONELA_ERR_ARG  # one pool


def evict_cfg(L, **change):
    f = dict(R=2, H_kv=2, d=64, dtype=1, page=16, pages=10, row_pages=4, dst_pages=6, dst_row_pages=2, keep=30,
             recent=8, device=0)
    f.update(change)
    return L._layers.onela_cache_evict_config(*[f[n] for n, _ in L._layers.onela_cache_evict_config._fields_])


def call_evict(L, cfg, bytes_=1 << 40, **change):
    a = dict(k=P, v=P, table=P, lengths=P, mass=P, dk=P, dv=3 * P, dt=P, dl=2 * P, dm=2 * P, kept=None, scratch=P)
    a.update(change)
    return L._lib.lib.onela_cache_evict(ctypes.addressof(cfg), *a.values(), bytes_, None, None)


@pytest.mark.parametrize("field,value", [
    ("R", 0), ("H_kv", 0), ("d", 0), ("d", 257), ("dtype", 5), ("page", 0), ("pages", 0), ("row_pages", 0),
    ("dst_pages", 0), ("dst_row_pages", 1), ("keep", 0), ("keep", 33), ("recent", -1), ("recent", 31),
    ("device", -1)])
def test_evict_refuses_bad_config(field, value):
    import linear_attention_beam_shared_b200 as L
    cfg = evict_cfg(L, **{field: value})
    assert call_evict(L, cfg) == L.ONELA_ERR_ARG
    assert L._lib.lib.onela_cache_evict_scratch_bytes(ctypes.addressof(cfg)) == 0


@pytest.mark.parametrize("change", [
    {n: None} for n in ("k", "v", "table", "lengths", "mass", "dk", "dv", "dt", "dl", "dm", "scratch")] + [
    dict(k=P + 1), dict(mass=P + 2), dict(scratch=P + 8), dict(dl=P), dict(dm=P), dict(dv=P)])
def test_evict_refuses_bad_pointers(change):
    import linear_attention_beam_shared_b200 as L
    assert call_evict(L, evict_cfg(L), **change) == L.ONELA_ERR_ARG
    assert call_evict(L, evict_cfg(L), 16) == L.ONELA_ERR_SCRATCH


def norm_cfg(L, **change):
    f = dict(N=4, y_stride=64, gate_stride=64, x_stride=64, D=64, group=32, y_dtype=0, dtype=1, act=2, device=0,
             alpha=1.0, eps=1e-6)
    f.update(change)
    return L._layers.onela_block_norm_config(*[f[n] for n, _ in L._layers.onela_block_norm_config._fields_])


def call_norm(L, cfg, **change):
    a = dict(y=P, gate=P, x=P, w_post=P, scale=P, w_pre=P, x_out=2 * P, n_out=3 * P)
    a.update(change)
    return L._lib.lib.onela_block_norm(ctypes.addressof(cfg), *a.values(), None)


@pytest.mark.parametrize("field,value", [
    ("N", -1), ("N", 1 << 31), ("D", 0), ("D", 32769), ("group", 0), ("group", 48), ("y_dtype", 3), ("dtype", -1),
    ("act", 3), ("act", 0), ("device", -1), ("eps", -1.0), ("eps", float("nan")), ("y_stride", 63),
    ("gate_stride", 0), ("x_stride", 63)])
def test_norm_refuses_bad_config(field, value):
    import linear_attention_beam_shared_b200 as L
    assert call_norm(L, norm_cfg(L, **{field: value})) == L.ONELA_ERR_ARG


@pytest.mark.parametrize("change", [
    dict(y=None, x=None), dict(y=None), dict(x_out=None, n_out=None), dict(w_pre=None), dict(n_out=None),
    dict(gate=None), dict(gate=P + 1), dict(w_post=P + 2), dict(y=P + 2),
    dict(n_out=3 * P, x_out=3 * P)])
def test_norm_refuses_bad_pointers(change):
    import linear_attention_beam_shared_b200 as L
    assert call_norm(L, norm_cfg(L), **change) == L.ONELA_ERR_ARG


def test_norm_refuses_in_place_over_spaced_rows_and_accepts_no_rows():
    import linear_attention_beam_shared_b200 as L
    assert call_norm(L, norm_cfg(L, x_stride=80), x_out=P) == L.ONELA_ERR_ARG
    assert call_norm(L, norm_cfg(L, N=0)) == L.ONELA_OK


def test_binding_refuses_cpu_tensors():
    import torch
    import linear_attention_beam_shared_b200 as L
    t = torch.zeros(1, 1, 1, 8)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        L.onela_paged_attention(t, t, t, i, i[0])
    with pytest.raises(ValueError):
        L.onela_cache_write(t, t, t, t, i, i[0])
    with pytest.raises(ValueError):
        L.onela_cache_evict(t, t, i, i[0], t[0], 1, 0, t, t, i, i[0], t[0])
    with pytest.raises(ValueError):
        L.onela_block_norm(y=t[0, 0])
    with pytest.raises(ValueError):
        L.onela_block_norm()


def test_binding_refuses_sizes_that_do_not_fit_their_fields():
    """2^32 + 5 must not pass for 5."""
    import linear_attention_beam_shared_b200 as L
    from linear_attention_beam_shared_b200 import _layers
    good = dict(R=1, W=1, H_q=4, H_kv=2, d=64, dtype="bf16", page=16, pages=10, row_pages=40)
    assert L.onela_paged_attention_scratch_bytes(**good) > 0
    for name in ("R", "W", "H_q", "pages", "row_pages"):
        with pytest.raises(ValueError):
            L.onela_paged_attention_scratch_bytes(**{**good, name: 2 ** 32 + good[name]})
    sizes = [1, 2, 64, 1, 16, 10, 40, 10, 40, 100, 9, 0]
    _layers._config(("test", tuple(sizes)), _layers.onela_cache_evict_config, sizes, None)
    for i in (9, 10):  # keep, recent
        bad = list(sizes)
        bad[i] += 2 ** 32
        with pytest.raises(ValueError):
            _layers._config(("test", tuple(bad)), _layers.onela_cache_evict_config, bad, None)


def test_attention_wait_policy_refuses_bad_bounds():
    import linear_attention_beam_shared_b200 as L
    f = L._lib.lib.onela_set_attention_wait_policy
    for limit, stall in ((999_999, 0), (10**10 + 1, 0), (10**9, -1), (10**9, 10)):
        assert f(limit, stall) == L.ONELA_ERR_ARG
        with pytest.raises(L.OnelaError):
            L.onela_set_attention_wait_policy(limit, stall)
    assert f(2_000_000_000, 0) == 0


def test_scratch_bytes_of_a_spaced_out_q():
    """A token stride that rules the tensor-core kernels out needs the general kernel's scratch."""
    import linear_attention_beam_shared_b200 as L
    sizes = (2, 64, 8, 2, 64, "bf16", 16, 100, 40)
    for mass in (False, True):
        general = L.onela_paged_attention_scratch_bytes(*sizes, want_mass=mass, kernel=L.ONELA_KERNEL_SIMT)
        dense = L.onela_paged_attention_scratch_bytes(*sizes, want_mass=mass)
        assert general != dense > 0
        assert L.onela_paged_attention_scratch_bytes(*sizes, want_mass=mass, q_stride=8 * 64 + 8) == dense
        assert L.onela_paged_attention_scratch_bytes(*sizes, want_mass=mass, q_stride=8 * 64 + 3) == general
    assert L.onela_paged_attention_scratch_bytes(*sizes, q_stride=8 * 64 - 1) == 0
    with pytest.raises(ValueError):
        L.onela_paged_attention_scratch_bytes(*sizes, q_stride=1 << 63)


def apart(n, first=1 << 40, step=1 << 36):
    """n addresses far from one another."""
    return [first + i * step for i in range(n)]


@pytest.mark.parametrize("out", ["o", "lse", "mass_out", "scratch"])
@pytest.mark.parametrize("over", ["lengths", "table", "bl", "bt"])
def test_attention_refuses_outputs_over_its_plan(out, over):
    """An output that begins inside, or reaches into, the lengths or a table."""
    import linear_attention_beam_shared_b200 as L
    cfg = attention(L, beam_page=1, beam_pages=9, beam_row_pages=5)
    names = ["q", "k", "v", "table", "lengths", "bk", "bv", "bt", "bl", "mass_out", "o", "lse", "scratch"]
    good = dict(zip(names, apart(len(names))))
    sizes = dict(o=2 * 3 * 8 * 64 * 2, lse=2 * 3 * 8 * 4, mass_out=2 * 2 * 640 * 4, scratch=256)
    for at in (good[over], good[over] - sizes[out] + (256 if out == "scratch" else 4)):
        a = dict(good, **{out: at})
        if out == "scratch":
            a["scratch"] -= a["scratch"] % 256
        assert call_attention(L, cfg, **a) == L.ONELA_ERR_ARG


@pytest.mark.parametrize("out,over", [(o, p) for o in ("dl", "dm", "dk", "dv", "kept", "scratch")
                                      for p in ("lengths", "mass", "table", "dt")] +
                         [("kept", p) for p in ("dl", "dm", "dk", "dv")] + [("scratch", p) for p in ("dl", "dm", "dk", "dv")])
def test_evict_refuses_outputs_over_its_plan(out, over):
    import linear_attention_beam_shared_b200 as L
    cfg = evict_cfg(L)
    names = ["k", "v", "table", "lengths", "mass", "dk", "dv", "dt", "dl", "dm", "kept", "scratch"]
    good = dict(zip(names, apart(len(names))))
    if out == "scratch":
        good["kept"] = None
    sizes = dict(dl=8, dm=2 * 2 * 32 * 4, dk=6 * 2 * 16 * 64 * 2, dv=6 * 2 * 16 * 64 * 2, kept=2 * 2 * 30 * 4, scratch=512)
    for at in (good[over], good[over] + (0 if out == "scratch" else 4) - sizes[out] + (256 if out == "scratch" else 0)):
        assert call_evict(L, cfg, **dict(good, **{out: at})) == L.ONELA_ERR_ARG
