"""The operators around a GDN layer and the handle's steps and folds on one
stream: each call sees what the calls before it wrote, however soon its kernel
may start.  Bitwise against the same chain with a device wait after every call."""
import pytest
import torch


pytestmark = pytest.mark.gpu


def draw(seed, R, H, d, W, T):
    """fp32 projections of every step (before their norms), gates, parents."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda")   # noqa: E731
    steps = []
    for t in range(T):
        par = torch.randint(0, 1 if t == 0 else W, (R, W), generator=gen, device="cuda", dtype=torch.int32)
        if t % 3 == 2:
            par[:] = t % W  # one ancestor for all: the folds have something to take
        steps.append(dict(q=rnd(R * W * H, d), k=rnd(R * W * H, d), v=rnd(R * W * H, d), g=-rnd(R * W, H).abs() * 0.1,
                          beta=torch.rand((R, W, H), generator=gen, device="cuda"), par=par))
    return rnd(R, H, d, d) * 0.1, steps


@pytest.mark.parametrize("T_max", [5, 16])
@pytest.mark.parametrize("captured", [False, True])
def test_step_after_a_fold_sees_the_norms_between(captured, T_max):
    """Fold, then per-head norms that write the next step's q, k, v and gate,
    then that step; all without flags."""
    import linear_attention_beam_shared_b200 as L
    R, H, d, W, T = 4, 16, 128, 256, 13
    S0, steps = draw(3, R, H, d, W, T)
    w = torch.ones(d, device="cuda") * d ** -0.5
    shape = (R, W, H, d)

    def run(wait, replay=False):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        dec = L.BeamDecoder(R, H, d, d, W, T_max, "f32", "bf16")
        q, k, v = (torch.zeros((R * W * H, d), dtype=torch.bfloat16, device="cuda") for _ in range(3))
        g = torch.zeros((R * W, H), device="cuda")
        outs = [torch.zeros(shape, device="cuda") for _ in range(T)]
        try:
            assert dec.kernel == L.ONELA_KERNEL_TC
            dec.set_prompt_state(S0)

            def chain():
                for t, s in enumerate(steps):
                    if t and t % 3 == 0:
                        dec.fold()
                        sync()
                    L.onela_block_norm(s["g"], alpha=0.5, x_out=g)
                    sync()
                    for y, x in ((s["v"], v), (s["k"], k), (s["q"], q)):  # q last: the kernel before the step
                        L.onela_block_norm(y, w_post=w, dtype="bf16", x_out=x)
                        sync()
                    dec.step(q.view(shape), k.view(shape), v.view(shape), g.view(R, W, H), s["beta"], s["par"], o=outs[t])
                    sync()
            if replay:
                stream = torch.cuda.Stream()
                stream.wait_stream(torch.cuda.current_stream())
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=stream):
                    chain()
                graph.replay()
                torch.cuda.synchronize()
                for o in outs:
                    o.zero_()
                graph.replay()
            else:
                chain()
            torch.cuda.synchronize()
            assert dec.status() == 0
            return outs
        finally:
            torch.cuda.synchronize()
            dec.close()

    want = run(True)
    assert all(torch.isfinite(o).all() for o in want) and float(want[-1].abs().max()) > 1e-3
    for _ in range(3):
        for t, (a, b) in enumerate(zip(want, run(False, captured))):
            assert torch.equal(a, b), f"step {t + 1}"


@pytest.mark.parametrize("captured", [False, True])
def test_flagged_steps_behind_a_norm_that_feeds_a_later_one(captured):
    """ONELA_FLAG_PDL: before step t a norm writes the q of step t + 1, so the
    kernel before each step produces no input of that step; k, gates and parents
    stay as they are throughout."""
    import linear_attention_beam_shared_b200 as L
    R, H, d, W, T = 4, 16, 128, 256, 12
    S0, steps = draw(4, R, H, d, W, T)
    w = torch.ones(d, device="cuda") * d ** -0.5
    shape = (R, W, H, d)
    for s in steps:
        s["k"], s["v"] = ((s[n] * d ** -0.5).bfloat16().view(shape) for n in ("k", "v"))
        s["g"] = s["g"].view(R, W, H)

    def run(wait, graph=False):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        dec = L.BeamDecoder(R, H, d, d, W, T, "f32", "bf16", flags=L.ONELA_FLAG_PDL)
        q = [torch.zeros((R * W * H, d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        outs = [torch.zeros(shape, device="cuda") for _ in range(T)]

        def chain():
            L.onela_block_norm(steps[0]["q"], w_post=w, dtype="bf16", x_out=q[0])
            sync()
            for t, s in enumerate(steps):
                if t + 1 < T and t % 2 == 0:  # before steps 1, 3, 5, ..: the q of the step after
                    L.onela_block_norm(steps[t + 1]["q"], w_post=w, dtype="bf16", x_out=q[(t + 1) % 2])
                    sync()
                dec.step(q[t % 2].view(shape), s["k"], s["v"], s["g"], s["beta"], s["par"], o=outs[t])
                sync()
                if t + 1 < T and t % 2 == 1:  # the q of the next step, and a norm of no step's behind it
                    L.onela_block_norm(steps[t + 1]["q"], w_post=w, dtype="bf16", x_out=q[(t + 1) % 2])
                    sync()
                    L.onela_block_norm(steps[0]["g"].view(R * W, H), alpha=2.0)
                    sync()
        try:
            dec.set_prompt_state(S0)
            torch.cuda.synchronize()
            if graph:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    chain()
                g.replay()
                torch.cuda.synchronize()
                for o in outs:
                    o.zero_()
                g.replay()
            else:
                chain()
            torch.cuda.synchronize()
            assert dec.status() == 0
            return outs
        finally:
            torch.cuda.synchronize()
            dec.close()

    want = run(True)
    for _ in range(3):
        for t, (a, b) in enumerate(zip(want, run(False, captured))):
            assert torch.equal(a, b), f"step {t + 1}"
