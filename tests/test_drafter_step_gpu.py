"""The drafter's step as it is used: the loss of the tokens that the target kept from the
drafter's hidden states, its gradients through autograd, and an orthogonalised update made of
the head's gradient; and the example that does so."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests._head64 import head64, hold  # noqa: E402
from tests._orth64 import bound, orth64  # noqa: E402
from tests._orth64 import hold as hold_matrix  # noqa: E402
from tests.test_example_gpu import _load  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def test_loss_gradients_and_update():
    vocab, dim, B, K = 900, 320, 24, 4
    g = torch.Generator(device="cuda").manual_seed(0)
    embed = torch.randn(vocab, dim, generator=g, device="cuda").requires_grad_()
    head = (torch.randn(vocab, dim, generator=g, device="cuda") / dim ** 0.5).requires_grad_()
    z = torch.randn(B, K + 1, vocab, generator=g, device="cuda")
    drafts = torch.randint(0, vocab, (B, K), generator=g, device="cuda").int()
    out = sv.specv_verify(z, z[:, :K], drafts, torch.ones(B, device="cuda"), torch.rand(B, K + 1, generator=g, device="cuda"))
    context = torch.cat([torch.zeros(B, 1, dtype=torch.int32, device="cuda"), drafts], 1).view(-1).long()
    targets = out["out_tokens"].view(-1)
    weights = (targets >= 0).float() / (targets >= 0).sum()
    loss = sv.head_loss(embed[context].bfloat16(), head.bfloat16(), targets, weights=weights)
    loss.sum().backward()
    want = head64(embed.detach()[context].bfloat16(), head.detach().bfloat16(), targets, weights=weights)
    hold(loss.detach(), want, "loss")
    hold(head.grad, want, "grad_head")  # (bf16, in fp32)
    # the embedding's rows: sums of the positions' gradients (autograd's own, in fp32)
    into = lambda x: torch.zeros(vocab, dim, dtype=torch.float64, device="cuda").index_add_(0, context, x)  # noqa: E731
    assert ((embed.grad.double() - into(want["grad_hidden"])).abs() <= 1.02 * into(want["grad_hidden_off"]) + 1e-30).all()
    o = sv.specv_orthogonalize(head.grad)
    assert o["row_status"] == 0
    hold_matrix(o["orthogonal"], orth64(head.grad)[0], bound(vocab, dim))


def test_captured_step():
    """Loss, gradients and update in one graph, on new inputs in the same buffers."""
    g = torch.Generator(device="cuda").manual_seed(1)
    make = lambda: (torch.randn(300, 128, generator=g, device="cuda").bfloat16(),  # noqa: E731
                    (torch.randn(700, 128, generator=g, device="cuda") / 8).bfloat16(),
                    torch.randint(-1, 700, (300,), generator=g, device="cuda").int())

    def step(h, W, t):
        o = sv.specv_head_loss(h, W, t, with_grad=True)
        return o["loss"], o["grad_hidden"], sv.specv_orthogonalize(o["grad_head"])["orthogonal"]

    static = make()
    step(*static)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*static)
    for _ in range(3):
        new = make()
        for x, y in zip(static, new):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(got, step(*new)))


@pytest.mark.parametrize("loss,update", [("tokens", "adam"), ("distill", "orthogonal"), ("tokens", "orthogonal")])
def test_example_runs(loss, update):
    accepted, losses = _load().run(rounds=12, batch=32, vocab=512, loss=loss, update=update)
    assert len(accepted) == len(losses) == 12
    assert all(0.0 <= a <= 4.0 for a in accepted) and all(x == x and abs(x) < 100 for x in losses)
