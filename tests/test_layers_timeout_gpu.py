"""Bounded waits of the attention's tensor-core kernels: a barrier that expects
an arrival which never comes makes the waits on it run out.  The kernels return,
report ONELA_STATUS_TIMEOUT and leave NaN where something is missing; the calls
after them are whole.  Nothing faults or hangs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def inputs(W, G, d, n, H=148, page=16):
    gen = torch.Generator(device="cuda").manual_seed(W + d)
    rows = -(-n // page)
    k, v = (torch.randn((rows, H, page, d), generator=gen, device="cuda").bfloat16() for _ in range(2))
    table = torch.randperm(rows, generator=gen, device="cuda").to(torch.int32)[None]
    q = torch.randn((1, W, H * G, d), generator=gen, device="cuda").bfloat16()
    return q, k, v, table, torch.tensor([n], dtype=torch.int32, device="cuda"), torch.zeros((1, H, rows * page), device="cuda")


def call(args, stall=0):
    import linear_attention_beam_shared_b200 as L
    q, k, v, table, lengths, mass = args
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(mass), torch.empty(q.shape[:3], device="cuda")
    try:
        if stall:
            L.onela_set_attention_wait_policy(2_000_000, stall)
        o = L.onela_paged_attention(q, k, v, table, lengths, mass=mass, mass_out=out, lse=lse, status=status)
        torch.cuda.synchronize()
    finally:
        L.onela_set_attention_wait_policy(2_000_000_000, 0)
    return o, lse, out, int(status)


# One CTA per head and row tile, 40 tiles of tokens each; the drawn weights take
# 3 or 11 tiles of query rows.
@pytest.mark.parametrize("W,G,d", [(40, 1, 64), (175, 4, 64), (44, 4, 128), (44, 4, 256)])
@pytest.mark.parametrize("stall", [1, 2, 3, 4, 5])
def test_attention_wait_runs_out(stall, W, G, d):
    import linear_attention_beam_shared_b200 as L
    args = inputs(W, G, d, 64 * 39 + 20)
    good = call(args)
    assert good[3] == 0 and all(torch.isfinite(x.float()).all() for x in good[:2])
    o, lse, mass, status = call(args, stall)
    assert status == L.ONELA_STATUS_TIMEOUT
    assert torch.isnan(o).all() and torch.isnan(lse).all() and torch.isnan(mass[:, :, :args[4].item()]).all()
    again = call(args)
    assert again[3] == 0 and all(torch.equal(a, b) for a, b in zip(again[:2], good[:2]))
    assert torch.equal(again[2][:, :, :args[4].item()], good[2][:, :, :args[4].item()])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("stall", [6, 7, 8, 9])
def test_drawn_weights_wait_runs_out(stall, d):
    import linear_attention_beam_shared_b200 as L
    args = inputs(175, 4, d, 500, H=5)
    good = call(args)
    o, lse, mass, status = call(args, stall)
    assert status == L.ONELA_STATUS_TIMEOUT
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
    assert torch.isnan(mass[:, :, :500]).all()
    again = call(args)
    assert again[3] == 0 and torch.equal(again[2][:, :, :500], good[2][:, :, :500])
