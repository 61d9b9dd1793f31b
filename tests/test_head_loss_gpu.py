"""specv_head_loss, its backward pass and head_loss against their definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests._head64 import head64, hold, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def check(h, W, t, **how):
    up = how.pop("up", None)
    want = head64(h, W, t, up=up, **how)
    if up is None:
        o = sv.specv_head_loss(h, W, t, with_grad=True, **how)
    else:
        o = sv.specv_head_loss(h, W, t, targets_only=True, **how)
        o.update(sv.specv_head_loss_backward(h, W, t, o["stats"], grad_loss=up, **how))
    assert (o["row_status"] == 0).all()
    hold(o["loss"], want, "loss")
    hold(o["stats"][:, 0], want, "lse")
    hold(o["stats"][:, 1], want, "nll")
    hold(o["grad_hidden"], want, "grad_hidden")
    hold(o["grad_head"], want, "grad_head")
    return o, want


SIZES = [(1, 64, 256), (1, 8, 1), (2, 16, 2), (1, 200, 1000), (5, 64, 127), (33, 128, 129), (64, 264, 513), (128, 64, 1024),
         (255, 72, 300), (256, 512, 2000), (257, 96, 777), (600, 1024, 5000), (1100, 40, 3333)]


@pytest.mark.parametrize("N,D,V", SIZES)
def test_loss_and_gradients(N, D, V):
    check(*inputs(N, D, V, seed=N))


@pytest.mark.parametrize("N,D,V", SIZES[::2])
def test_backward_with_upstream(N, D, V):
    h, W, t = inputs(N, D, V, seed=N + 1)
    check(h, W, t, up=torch.rand(N, device="cuda") + 0.5, scale=0.7)


@pytest.mark.parametrize("N", [40, 400])
@pytest.mark.parametrize("D,pad,off", [(65, 0, 0), (64, 3, 0), (64, 8, 0), (64, 0, 1), (31, 2, 3), (7, 1, 0), (1, 0, 0),
                                       (65, 7, 0), (31, 1, 0), (300, 4, 8), (1, 7, 0)])
def test_strides_and_alignments(N, D, pad, off):
    h, W, t = inputs(N, D, 500, seed=D, pad=pad, off=off)
    o, want = check(h, W, t)
    # gradients into rows with gaps, which stay as they are
    for gap in (5, 8 - D % 8, 16 - D % 8):
        room = [torch.full((x.shape[0], D + gap), 7.0, dtype=torch.bfloat16, device="cuda") for x in (h, W)]
        sv.specv_head_loss(h, W, t, grad_hidden=room[0][:, :D], grad_head=room[1][:, :D])
        assert torch.equal(room[0][:, :D], o["grad_hidden"]) and torch.equal(room[1][:, :D], o["grad_head"])
        assert all((x[:, D:] == 7).all() for x in room)


@pytest.mark.parametrize("N,D,V", [(8200, 16, 70000), (300, 264, 9000)])
def test_pieces_of_the_vocabulary(N, D, V):
    """More weights than a call keeps, and a backward pass in several pieces."""
    h, W, t = inputs(N, D, V, seed=3)
    check(h, W, t)
    check(h, W, t, up=torch.rand(N, device="cuda"))


def masked(N, D, V, seed=0):
    """Rows without a target or weight, which hold NaN and infinities."""
    h, W, t = inputs(N, D, V, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kind = torch.randint(0, 4, (N,), generator=g, device="cuda")
    t[kind == 1] = -1
    w = torch.rand(N, generator=g, device="cuda") + 0.5
    w[kind == 2] = 0.0
    h[kind == 1] = float("nan")
    h[kind == 2] = float("inf")
    return h, W, t, w


@pytest.mark.parametrize("N", [1, 7, 64, 256, 257, 700, 2000])
def test_rows_that_are_left_out(N):
    h, W, t, w = masked(N, 128, 777, seed=N)
    for up in (None, torch.rand(N, device="cuda") - 0.5):
        o, _ = check(h, W, t, weights=w, **({} if up is None else dict(up=up)))
    out = (t < 0) | (w == 0)
    assert (o["loss"][out] == 0).all() and (o["stats"][out] == 0).all() and (o["grad_hidden"][out] == 0).all()


@pytest.mark.parametrize("N", [1, 45, 200, 700])
def test_log_sum_exp_of_rows_without_a_target(N):
    h, W, t = inputs(N, 136, 999, seed=N)
    t[::3] = -1
    w = torch.ones(N, device="cuda")
    w[1::5] = 0
    o = sv.specv_head_loss(h, W, t, weights=w, scale=1.25)
    want = head64(h, W, t.clamp_min(0), weights=w, scale=1.25)
    hold(o["stats"][:, 0], want, "lse")
    none = t < 0
    assert (o["row_status"] == 0).all() and (o["loss"][none] == 0).all() and (o["stats"][none, 1] == 0).all()
    only = sv.specv_head_loss(h, W, t, weights=w, scale=1.25, targets_only=True)
    assert (only["stats"][none] == 0).all() and torch.equal(only["stats"][~none], o["stats"][~none])
    h[0] = float("nan")
    o = sv.specv_head_loss(h, W, t, weights=w)
    assert o["row_status"][0] == 0 and o["stats"][0, 0].isnan() and o["loss"][0] == 0


@pytest.mark.parametrize("N", [5, 300])
def test_no_row_counts(N):
    h, W, t = inputs(N, 64, 300)
    t.fill_(-1)
    h.fill_(float("nan"))
    o = sv.specv_head_loss(h, W, t, with_grad=True)
    assert all((o[k] == 0).all() for k in ("loss", "stats", "grad_hidden", "grad_head", "row_status"))
    b = sv.specv_head_loss_backward(h, W, t, o["stats"])
    assert (b["grad_hidden"] == 0).all() and (b["grad_head"] == 0).all()


def test_no_rows():
    W = torch.randn(100, 64, device="cuda").bfloat16()
    h, t = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    o = sv.specv_head_loss(h, W, t, with_grad=True)
    assert o["loss"].shape == (0,) and (o["grad_head"] == 0).all()
    room = torch.full((100, 70), 7.0, dtype=torch.bfloat16, device="cuda")
    sv.specv_head_loss_backward(h, W, t, o["stats"], grad_head=room[:, :64])
    assert (room[:, :64] == 0).all() and (room[:, 64:] == 7).all()


@pytest.mark.parametrize("N", [20, 400])
def test_bad_rows_are_flagged_alone(N):
    h, W, t = inputs(N, 72, 500, seed=1)
    want = head64(h, W, t)
    good = torch.ones(N, dtype=torch.bool, device="cuda")
    bad = {3: (500, sv.ROW_BAD_TOKEN), 5: (-2, sv.ROW_BAD_TOKEN), 8: (float("nan"), sv.ROW_NONFINITE),
           9: (float("inf"), sv.ROW_NONFINITE), 10: (float("-inf"), sv.ROW_NONFINITE), N - 1: (3.3e38, sv.ROW_NONFINITE)}
    for r, (x, s) in bad.items():
        good[r] = False
        if s == sv.ROW_BAD_TOKEN:
            t[r] = x
        elif x == 3.3e38:
            h[r] = x  # finite, but its logits are not
        else:
            h[r, 17] = x
    o = sv.specv_head_loss(h, W, t, with_grad=True)
    b = sv.specv_head_loss_backward(h, W, t, o["stats"])
    for r, (_, s) in bad.items():
        assert o["row_status"][r] == s, r
    assert (o["row_status"][good] == 0).all()
    assert (o["loss"][~good] == 0).all() and o["stats"][~good].isnan().all()
    clean = head64(h.nan_to_num(0, 0, 0) * good[:, None], W, torch.where(good, t, -1))
    for x in (o, b):
        assert (x["grad_hidden"][~good] == 0).all()
        hold(x["grad_hidden"][good], {k: v[good] for k, v in clean.items() if k.startswith("grad_hidden")}, "grad_hidden")
        hold(x["grad_head"], clean, "grad_head")
    hold(o["loss"][good], {k: v[good] for k, v in want.items() if k.startswith("loss")}, "loss")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_head_that_is_not_finite_flags_every_row(bad):
    h, W, t = inputs(30, 64, 400)
    W[399, 5] = bad
    o = sv.specv_head_loss(h, W, t, with_grad=True)
    assert (o["row_status"] == sv.ROW_NONFINITE).all()
    assert (o["loss"] == 0).all() and (o["grad_hidden"] == 0).all() and (o["grad_head"] == 0).all()


@pytest.mark.parametrize("size", [1e-3, 1.0, 30.0])
def test_sizes_of_logits(size):
    """From flat rows to rows whose loss is 0 or hundreds."""
    h, W, t = inputs(270, 256, 1500, seed=4, lean=0.0)
    h = (h * size).bfloat16()
    h[::2] += (size * W[t[::2].long()] * 4).bfloat16()
    check(h, W, t)
    check(h, W, t, up=torch.ones(270, device="cuda"))


def test_long_hidden_states():
    """Sums over more than one chunk of D, with a tail."""
    check(*inputs(130, 5003, 600, seed=5))
    check(*inputs(300, 2056, 600, seed=6))


@pytest.mark.parametrize("N", [45, 600])
def test_one_gradient_alone_and_calls_again(N):
    h, W, t = inputs(N, 200, 3000, seed=7)
    o = sv.specv_head_loss(h, W, t, with_grad=True)
    again = sv.specv_head_loss(h, W, t, with_grad=True)
    gh = sv.specv_head_loss(h, W, t, grad_hidden=torch.empty_like(h))
    gW = sv.specv_head_loss(h, W, t, grad_head=torch.empty_like(W))
    assert "grad_head" not in gh and "grad_hidden" not in gW
    for k in o:
        assert torch.equal(o[k], again[k]), k
    assert torch.equal(gh["grad_hidden"], o["grad_hidden"]) and torch.equal(gW["grad_head"], o["grad_head"])
    b = sv.specv_head_loss_backward(h, W, t, o["stats"])
    for k, x in (("grad_hidden", h), ("grad_head", W)):
        alone = sv.specv_head_loss_backward(h, W, t, o["stats"], **{k: torch.empty_like(x)})
        assert list(alone) == [k] and torch.equal(alone[k], b[k])


def test_differentiable():
    h, W, t, w = masked(300, 96, 1000, seed=8)
    up = torch.rand(300, device="cuda")
    want = head64(h, W, t, weights=w, up=up, scale=1.5)
    x, y = h.clone().requires_grad_(), W.clone().requires_grad_()
    loss = sv.head_loss(x, y, t, weights=w, scale=1.5)
    loss.backward(up)
    hold(loss.detach(), want, "loss")
    hold(x.grad, want, "grad_hidden")
    hold(y.grad, want, "grad_head")
    # one leaf alone, and a broadcast upstream gradient
    x = h.clone().requires_grad_()
    sv.head_loss(x, W, t, weights=w).sum().backward()
    hold(x.grad, head64(h, W, t, weights=w), "grad_hidden")
    y = W.clone().requires_grad_()
    (sv.head_loss(h, y, t, weights=w) * 2).sum().backward()
    hold(y.grad, head64(h, W, t, weights=w, up=torch.full((300,), 2.0, device="cuda")), "grad_head")


def test_gradient_against_differences():
    """Steps of hidden that bf16 holds exactly.  A central difference of a row's loss along a
    direction is off by step^2 / 6 of a third derivative: the third central moment of the
    logits' slopes, at most S^3 for slopes within [-S, S]."""
    h, W, t = inputs(64, 64, 512, seed=9)
    h = (h.float().clamp(-1.9, 1.9) * 32).round().div(32).bfloat16()
    v = torch.randint(0, 2, h.shape, device="cuda").bfloat16() * 2 - 1
    step = 1.0 / 64
    assert torch.equal((h + step * v).float(), h.float() + step * v.float())
    slopes = (v.double() @ W.double().T).abs().amax(1)
    losses = [sv.specv_head_loss(h + s * step * v, W, t)["loss"].double().sum() for s in (1, -1)]
    o = sv.specv_head_loss(h, W, t, with_grad=True)
    want = (losses[0] - losses[1]) / (2 * step)
    got = (o["grad_hidden"].double() * v.double()).sum()
    # the losses' own errors, and the gradient's
    exact = head64(h, W, t)
    bound = (slopes ** 3).sum() * step ** 2 / 6 + exact["loss_off"].sum() / step + exact["grad_hidden_off"].sum()
    assert abs(got - want) <= bound, (got, want, bound)


def test_graphs_streams_and_workspaces():
    a, b = inputs(40, 128, 2000, seed=10), inputs(400, 128, 2000, seed=11)
    direct = [sv.specv_head_loss(*x, with_grad=True) for x in (a, b)]
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = sv.specv_head_loss(*x, with_grad=True)
            o.update({"again_" + k: v for k, v in sv.specv_head_loss_backward(*x, o["stats"]).items()})
        graphs.append(g)
        outs.append(o)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for o, d in zip(outs, direct):
        assert all(torch.equal(o[k], d[k]) for k in d)
    # new inputs in the same buffers
    c = inputs(40, 128, 2000, seed=12)
    for x, y in zip(a, c):
        x.copy_(y)
    graphs[0].replay()
    torch.cuda.synchronize()
    want = sv.specv_head_loss(*c, with_grad=True)
    assert all(torch.equal(outs[0][k], want[k]) for k in want)
    # two streams at once, each call with its own workspace
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [sv.specv_head_loss(*x, with_grad=True, stream=s[k % 2]) for k, x in enumerate((a, b) * 3)]
    torch.cuda.synchronize()
    for k, o in enumerate(got):
        d = want if k % 2 == 0 else direct[1]
        assert all(torch.equal(o[n], d[n]) for n in d)


def test_workspace_of_the_size_asked_for():
    import ctypes
    for N, pad in ((33, 0), (300, 3)):
        h, W, t = inputs(N, 65, 700, pad=pad)
        args = sv._head_args(h, W, t, 1.0, None, torch.empty(N, 65, dtype=h.dtype, device="cuda"),
                             torch.empty(700, 65, dtype=h.dtype, device="cuda"))
        need = sv.load_library().specv_head_workspace_bytes(ctypes.byref(args))
        room = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        o = sv.specv_head_loss(h, W, t, with_grad=True, workspace=room[:need])
        assert (room[need:] == 0x5a).all()
        with pytest.raises(sv.SpecvError):
            sv.specv_head_loss(h, W, t, with_grad=True, workspace=room[:need - 1])
        assert all(torch.equal(o[k], v) for k, v in sv.specv_head_loss(h, W, t, with_grad=True).items())
        sv.specv_head_loss_backward(h, W, t, o["stats"], workspace=room[:need])
        assert (room[need:] == 0x5a).all()


@pytest.mark.parametrize("N,D,V", [(70001, 16, 700), (3, 24, 1000003), (64, 64, 300000), (200, 320, 50000), (5, 200, 200000)])
def test_many_rows_and_many_tokens(N, D, V):
    check(*inputs(N, D, V, seed=13))


def test_offsets_past_32_bits():
    """A head of 2.3 x 10^9 elements: the loss over all of it, gradients of its last rows."""
    N, D, V = 2, 16384, 140003
    g = torch.Generator(device="cuda").manual_seed(14)
    W = torch.empty(V, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g).mul_(2.0 / D ** 0.5)
    h = torch.randn(N, D, generator=g, device="cuda").bfloat16()
    t = torch.tensor([V - 1, 5], dtype=torch.int32, device="cuda")
    o = sv.specv_head_loss(h, W, t, with_grad=True)
    b = sv.specv_head_loss_backward(h, W, t, o["stats"])
    z = torch.cat([h.double() @ W[k:k + 20000].double().T for k in range(0, V, 20000)], 1)
    logp = torch.log_softmax(z, 1)
    # a sum over 16384 in 256s: (16 + 2) roundings of 2^-23 of the products' absolute sum, and 64 of chunks
    size = h.double().abs().sum(1) * W.abs().amax().double()
    assert ((o["loss"].double() + logp.gather(1, t.long()[:, None])[:, 0]).abs() <= 2 * 82 * 2.0 ** -23 * size).all()
    d = logp.exp()
    d[torch.arange(N), t.long()] -= 1
    last = slice(V - 300, V)
    want = d[:, last].T @ h.double()
    scale = d[:, last].abs().T @ h.double().abs()
    for x in (o, b):  # dz and the result rounded to bf16, the weights to fp16; logits off as above
        off = (x["grad_head"][last].double() - want).abs()
        assert (off <= (2.0 ** -8 + 2.0 ** -11 + 2 * 82 * 2.0 ** -23 * size.max()) * scale + 2.0 ** -8 * want.abs() + 1e-30).all()
        part = torch.cat([d[:, k:k + 20000] @ W[k:k + 20000].double() for k in range(0, V, 20000)]).view(-1, N, D).sum(0)
        bound = torch.cat([d[:, k:k + 20000].abs() @ W[k:k + 20000].double().abs() for k in range(0, V, 20000)]).view(-1, N, D).sum(0)
        off = (x["grad_hidden"].double() - part).abs()
        assert (off <= (2.0 ** -8 + 2.0 ** -11 + 2 * 82 * 2.0 ** -23 * size.max() + (V / 16 + 34) * 2.0 ** -23) * bound
                + 2.0 ** -8 * part.abs()).all()
