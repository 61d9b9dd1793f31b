"""specv_orthogonalize against its steps in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests._orth64 import bound, hold, orth64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def matrix(shape, kind="random", seed=0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    small = min(shape[-2:])
    if kind == "falling":  # singular values that fall as 1 / k
        q, _ = torch.linalg.qr(torch.randn(shape[-2], shape[-2], generator=g, device="cuda", dtype=torch.float64))
        r, _ = torch.linalg.qr(torch.randn(shape[-1], shape[-1], generator=g, device="cuda", dtype=torch.float64))
        x = (q[:, :small] * (1.0 / torch.arange(1, small + 1, device="cuda"))) @ r[:small]
    if kind == "low rank":
        k = max(1, small // 16)
        x = torch.randn(*shape[:-1], k, generator=g, device="cuda") @ torch.randn(*shape[:-2], k, shape[-1], generator=g, device="cuda")
        x = x + 0.05 * torch.randn(*shape, generator=g, device="cuda")
    return x.to(dtype)


def check(G, **how):
    want, norm = orth64(G, **how)
    o = sv.specv_orthogonalize(G, **how)
    assert (o["row_status"] == 0).all()
    # squares of entries, sums of up to 2^24 of them in fp32 in several hundred parts
    assert ((o["norm"].double() - norm).abs() <= 2.0 ** -17 * norm).all()
    hold(o["orthogonal"], want, bound(*G.shape[-2:], how.get("steps", 5)))
    return o


SHAPES = [(1, 1), (1, 7), (2, 2), (3, 300), (64, 64), (65, 127), (128, 512), (255, 257), (256, 256), (300, 200), (512, 100),
          (700, 1111), (1030, 520), (2000, 64),
          (128, 128), (128, 129), (127, 2048), (2048, 128), (128, 2049), (2500, 33), (1, 2048), (130, 1), (16, 1025),
          (100, 9001), (250, 12000), (6000, 90), (600, 9000), (4001, 300)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_random(shape, dtype):
    check(matrix(shape, dtype=dtype, seed=shape[0]))


@pytest.mark.parametrize("shape", [(128, 512), (300, 200), (700, 1111)])
@pytest.mark.parametrize("kind", ["falling", "low rank"])
def test_spectra(shape, kind):
    check(matrix(shape, kind))


@pytest.mark.parametrize("shape", [(3, 64, 64), (5, 100, 333), (4, 333, 100), (24, 130, 130), (2, 1, 9), (200, 40, 90), (30, 600, 128), (2, 60, 5000), (3, 300, 4000)])
def test_batches(shape):
    G = matrix(shape, dtype=torch.bfloat16)
    G *= torch.logspace(-6, 6, shape[0], device="cuda").to(G.dtype)[:, None, None]
    o = check(G)
    for k in (0, shape[0] - 1):
        assert torch.equal(o["orthogonal"][k], sv.specv_orthogonalize(G[k])["orthogonal"])


def test_zero_and_not_finite_matrices():
    G = matrix((4, 100, 300))
    G[1] = 0
    G[2, 99, 299] = float("nan")
    G[3, 0, 0] = float("-inf")
    o = sv.specv_orthogonalize(G)
    assert o["row_status"].tolist() == [0, 0, sv.ROW_NONFINITE, sv.ROW_NONFINITE]
    assert (o["orthogonal"][1:] == 0).all() and o["norm"][1] == 0 and o["norm"][2:].isnan().all()
    assert torch.equal(o["orthogonal"][0], sv.specv_orthogonalize(G[0])["orthogonal"])


@pytest.mark.parametrize("shape", [(70, 130), (300, 513)])
def test_scale_does_not_matter(shape):
    """Powers of two give the same bits, from sums of squares that fp32 has no room for to numbers
    below its normal ones (whose own digits are fewer: they are compared with the exact steps)."""
    G = matrix(shape, dtype=torch.bfloat16).float()
    first = sv.specv_orthogonalize(G)
    for k in (-90, -20, 20, 60, 120):
        o = sv.specv_orthogonalize(torch.ldexp(G, torch.tensor(k, device="cuda")))
        assert torch.equal(o["orthogonal"], first["orthogonal"]), k
        assert o["norm"] == torch.ldexp(first["norm"], torch.tensor(k, device="cuda")), k
    small = G * 2.0 ** -70 * 2.0 ** -65
    hold(sv.specv_orthogonalize(small)["orthogonal"], orth64(small)[0], bound(*shape))


def test_one_huge_entry():
    G = matrix((300, 600)) * 1e-4
    G[7, 9] = 1e20
    check(G)


@pytest.mark.parametrize("shape", [(90, 33), (300, 517), (517, 300), (64, 72)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides(shape, dtype):
    """(Rows with gaps are summed in other parts: the norm's last digit may differ.)"""
    m, n = shape
    G = matrix((3, m, n), dtype=dtype)
    exact, _ = orth64(G)
    for pad, off in ((0, 1), (3, 0), (8, 0), (5, 2)):
        room = torch.full((3 * (m + 1) * (n + pad) + off,), float("nan"), dtype=dtype, device="cuda")
        x = room[off:].view(3, m + 1, n + pad)[:, :m, :n]
        x.copy_(G)
        want = sv.specv_orthogonalize(x)["orthogonal"]
        hold(want, exact, bound(m, n))
        out = torch.full((3, m + 2, n + pad + 1), 7.0, dtype=torch.bfloat16, device="cuda")
        sv.specv_orthogonalize(x, out=out[:, 1:m + 1, :n])
        assert torch.equal(out[:, 1:m + 1, :n], want), (pad, off)
        assert (out[:, 0] == 7).all() and (out[:, m + 1] == 7).all() and (out[..., n:] == 7).all()


def test_in_place():
    G = matrix((2, 130, 264), dtype=torch.bfloat16)
    want = sv.specv_orthogonalize(G)["orthogonal"]
    assert sv.specv_orthogonalize(G, out=G)["orthogonal"] is G and torch.equal(G, want)


def test_shared_update():
    """A matrix that is broadcast over the batch."""
    G = matrix((40, 60))
    o = sv.specv_orthogonalize(G.contiguous()[None].repeat(2, 1, 1))["orthogonal"]
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], sv.specv_orthogonalize(G)["orthogonal"])


@pytest.mark.parametrize("steps", [1, 2, 8])
def test_steps(steps):
    check(matrix((300, 400)), steps=steps)


def test_other_coefficients():
    """The steps whose limit is exact, X (15 - 10 S + 3 S S) / 8: errors of a step a third of
    the default's, and no step amplifies by more than 15/8."""
    G = matrix((260, 300))
    o = check(G, steps=12, coefficients=(1.875, -1.25, 0.375))["orthogonal"].double()
    s = torch.linalg.svdvals(o)
    assert (s[:130] - 1).abs().max() < 2.0 ** -7


@pytest.mark.parametrize("shape", [(200, 80), (700, 500), (100, 100)])
def test_transposed(shape):
    G = matrix(shape)
    a, b = (sv.specv_orthogonalize(x)["orthogonal"] for x in (G, G.T.contiguous()))
    hold(a, b.T.double(), 2 * bound(*shape))


def test_graphs_and_streams():
    a, b = matrix((100, 300), dtype=torch.bfloat16), matrix((3, 300, 290))
    direct = [sv.specv_orthogonalize(x)["orthogonal"] for x in (a, b)]
    graphs, outs = [], []
    for x in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sv.specv_orthogonalize(x)["orthogonal"])
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, d) for o, d in zip(outs, direct))
    s = [torch.cuda.Stream() for _ in range(2)]
    got = [sv.specv_orthogonalize(x, stream=s[k % 2])["orthogonal"] for k, x in enumerate((a, b) * 3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, direct[k % 2]) for k, o in enumerate(got))


@pytest.mark.parametrize("shape", [(1, 130, 200), (2, 300, 333)])
def test_workspace_of_the_size_asked_for(shape):
    G = matrix(shape)
    need = sv.load_library().specv_orthogonalize_workspace_bytes(*shape)
    room = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    o = sv.specv_orthogonalize(G, workspace=room[:need])
    assert (room[need:] == 0x5a).all()
    assert torch.equal(o["orthogonal"], sv.specv_orthogonalize(G)["orthogonal"])
    with pytest.raises(sv.SpecvError):
        sv.specv_orthogonalize(G, workspace=room[:need - 1])


@pytest.mark.parametrize("B,m,n", [(33000, 256, 256), (17000, 128, 1000), (140000, 130, 120)])
def test_offsets_past_32_bits(B, m, n):
    """Batches of more than 2^31 elements: the last matrices as if they were alone."""
    G = torch.empty(B, m, n, dtype=torch.bfloat16, device="cuda")
    if B > 65535:  # (more matrices than a call takes)
        with pytest.raises(sv.SpecvError):
            sv.specv_orthogonalize(G)
        return
    G.normal_(generator=torch.Generator(device="cuda").manual_seed(15))
    o = sv.specv_orthogonalize(G)
    assert (o["row_status"] == 0).all()
    for k in (0, B // 2, B - 1):
        alone = sv.specv_orthogonalize(G[k])
        hold(o["orthogonal"][k], orth64(G[k])[0], bound(m, n))
        hold(alone["orthogonal"], orth64(G[k])[0], bound(m, n))
