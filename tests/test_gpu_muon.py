"""GPU tests of the Muon step against the 64-bit definition.

Tolerance of X (2-norm, relative).  Each product's factors are exact to 2^-22 and its sums to
fp32; what the steps do with such errors was emulated on the host with operands rounded so:
below 5e-6 for matrices of independent elements, whose singular values lie close together, and
5e-5 for the hardest spectra tried (one large value and all others 1e-2 to 1e-8 of it, geometric
ones).  Four times that is allowed for the sums, which the emulation took as exact."""
import math

import pytest
import torch

import moe_expert_ffn_top_gb300 as m
import post_ref as ref
from post_ref import U32
from train_ops_ref import TINY_OF, UNIT

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
COEFS = (3.4445, -4.7750, 2.0315)
EASY, HARD = 4 * 5e-6, 4 * 5e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    yield


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _orthogonalised(u, **kw):
    """X of u, as the weights of a step from 0 with lr = -1 and no momentum."""
    p, mom = torch.zeros_like(u), torch.zeros_like(u)
    t = m.MuonTensors([dict(p=p, g=u, m=mom, lr=-1.0, scale=1.0)])
    m.moe_lora_muon_step(t, **dict(dict(momentum=0.0, nesterov=False), **kw))
    assert m.moe_lora_muon_get_error(t) == 0
    assert torch.equal(mom, u)
    return p


def _off(got, want):
    """Largest relative 2-norm of the difference over the matrices."""
    n = (got.double() - want).flatten(-2).norm(dim=-1) / want.flatten(-2).norm(dim=-1)
    return float(n.max())


SHAPES = [  # leading axes and matrix
    (1, 1), (1, 7), (5, 1), (2, 3), (8, 64), (64, 8), (3, 16, 256), (9, 256, 16), (16, 256), (128, 128), (128, 4096), (4096, 128),
    (5, 128, 700), (7, 768, 8), (33, 8, 768), (20, 24, 300), (20, 300, 24), (11, 13, 77), (11, 77, 13), (4, 100, 1001), (4, 1001, 100),
    (2, 3, 64, 130), (300, 2, 2), (3, 127, 128), (2, 90, 10000), (130, 31, 33)]


@pytest.mark.parametrize("shape", SHAPES)
def test_orthogonalised(shape):
    u = torch.randn(*shape, generator=_gen(sum(shape)), device="cuda")
    assert _off(_orthogonalised(u), ref.newton_schulz(u, 5, COEFS, 1e-7)) <= (EASY if max(shape[-2:]) >= 4 * min(shape[-2:]) else HARD)


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("shape", [(3, 40, 200), (5, 200, 64)])
def test_steps_and_coefficients(steps, shape):
    u = torch.randn(*shape, generator=_gen(steps), device="cuda")
    for coefs in (COEFS, (1.5, -0.5, 0.0), (15 / 8, -10 / 8, 3 / 8)):
        assert _off(_orthogonalised(u, steps=steps, coefs=coefs), ref.newton_schulz(u, steps, coefs, 1e-7)) <= EASY


@pytest.mark.parametrize("short,long_", [(128, 1024), (16, 256), (64, 2048)])
def test_spectra(short, long_):
    g = _gen(short)
    U = torch.linalg.qr(torch.randn(short, short, generator=g, device="cuda", dtype=torch.float64))[0]
    V = torch.linalg.qr(torch.randn(long_, short, generator=g, device="cuda", dtype=torch.float64))[0]
    one = torch.ones(short, dtype=torch.float64, device="cuda")
    few = torch.where(torch.arange(short, device="cuda") < 4, 1.0, 0.01).double()
    for sig in (one, torch.linspace(0.5, 1.5, short, device="cuda").double(), few, torch.where(torch.arange(short, device="cuda") < 1, 1.0, 1e-3).double(),
                torch.logspace(0, -4, short, device="cuda").double(), torch.logspace(0, -8, short, device="cuda").double()):
        u = ((U * sig) @ V.T).float()
        want = ref.newton_schulz(u, 5, COEFS, 1e-7)
        assert _off(_orthogonalised(u), want) <= HARD
        assert _off(_orthogonalised(u.T.contiguous()), want.T) <= HARD


def test_sizes_of_very_different_matrices():
    """Matrices of one tile do not see each other's size, zeros or bad elements."""
    u = torch.randn(16, 16, 200, generator=_gen(1), device="cuda")
    size = 10.0 ** torch.linspace(-12, 12, 16, device="cuda")
    u = u * size[:, None, None]
    u[3] = 0
    want = ref.newton_schulz(u, 5, COEFS, 1e-7)
    bad = u.clone()
    bad[5, 2, 100], bad[9, 15, 199], bad[10, 0, 0] = math.nan, math.inf, -math.inf
    bad[11] *= 1e12  # a norm whose square passes fp32's range
    keep = [i for i in range(16) if i not in (3, 5, 9, 10, 11)]
    for x in (bad, bad.mT.contiguous()):
        p = torch.zeros_like(x)
        mom = torch.zeros_like(x)
        t = m.MuonTensors([dict(p=p, g=x, m=mom, lr=-1.0, scale=1.0)])
        m.moe_lora_muon_step(t, momentum=0.0, nesterov=False)
        got = p if x is bad else p.mT
        assert _off(got[keep], want[keep]) <= EASY
        assert (got[3] == 0).all()
        assert all(torch.isnan(got[i]).all() for i in (5, 9, 10, 11))
    for scale in (1e-25, 0.0):  # nothing left of the norm
        assert (_orthogonalised(torch.full((4, 8), scale, device="cuda")) == 0).all()


@pytest.mark.parametrize("shape", [(6, 128, 520), (6, 520, 128), (40, 12, 36), (40, 36, 12), (9, 13, 70), (9, 70, 13)])
@pytest.mark.parametrize("pdt,gdt,master,nesterov", [(F32, F32, False, True), (BF, F32, True, False), (HF, HF, True, True), (BF, BF, False, True),
                                                    (F32, BF, False, False), (HF, F32, False, True)])
def test_step(shape, pdt, gdt, master, nesterov):
    """Momentum, weights, masters and their types over three steps; what lies around them stays."""
    g = _gen(sum(shape))
    n = math.prod(shape)

    def inside(dtype, value):  # a tensor inside a buffer with a guard on each side
        buf = torch.full((n + 128,), 7.0, dtype=dtype, device="cuda")
        buf[64:64 + n] = value.reshape(-1).to(dtype)
        return buf, buf[64:64 + n].view(shape)
    w0 = 0.05 * torch.randn(*shape, generator=g, device="cuda")
    pb, p = inside(pdt, w0)
    mb, mom = inside(F32, 0.1 * torch.randn(*shape, generator=g, device="cuda"))
    wb, wm = inside(F32, w0)
    grad = torch.empty(shape, dtype=gdt, device="cuda")
    lr, wd, scale = 0.01, 0.1, 1.7
    gs = torch.full((1,), 0.6, device="cuda")
    t = m.MuonTensors([dict(p=p, g=grad, m=mom, master=wm if master else None, lr=lr, weight_decay=wd, scale=scale)])
    for _ in range(3):
        grad.copy_(0.2 * torch.randn(*shape, generator=g, device="cuda"))
        src = (wm if master else p).clone()
        want_w, want_m, x = ref.muon(src, mom, grad, float(gs), 0.9, nesterov, 5, COEFS, 1e-7, lr, wd, scale)
        msize = 0.9 * mom.double().abs() + 0.1 * (grad.double() * float(gs)).abs()
        m.moe_lora_muon_step(t, momentum=0.9, nesterov=nesterov, grad_scale=gs)
        assert ((mom.double() - want_m).abs() <= 4 * U32 * msize).all()
        got = wm if master else p
        # elements: the 2-norm's bound for the whole matrix, every element being at most 2 in these
        err = lr * scale * HARD * x.flatten(-2).norm(dim=-1)[..., None, None] + 4 * U32 * (want_w.abs() + lr * scale * x.abs())
        unit = U32 if master else UNIT[pdt]
        assert ((got.double() - want_w).abs() <= err * (1 + unit) + unit * want_w.abs() + TINY_OF[F32 if master else pdt]).all()
        if master:
            assert torch.equal(p, wm.to(pdt))
    for b in (pb, mb) + ((wb,) if master else ()):
        assert (b[:64] == 7.0).all() and (b[64 + n:] == 7.0).all()
    if not master:
        assert torch.equal(wb[64:64 + n].view(shape), w0)
    assert m.moe_lora_muon_get_error(t) == 0


def test_many_tensors_graph_and_stream():
    """More tensors than one launch takes, empty ones among them; equal bits alone, on a side stream and replayed."""
    g = _gen(9)
    shapes = [[(2, 8, 40), (3, 70, 16), (1, 128, 256), (0, 4, 5), (17, 5)][i % 5] for i in range(300)]
    make = lambda: [dict(p=torch.zeros(s, device="cuda"), g=gr, m=torch.zeros(s, device="cuda"), lr=-1.0, scale=1.0) for s, gr in zip(shapes, grads)]  # noqa: E731
    grads = [torch.randn(*s, generator=g, device="cuda") for s in shapes]
    a = m.MuonTensors(make())
    m.moe_lora_muon_step(a, momentum=0.5)
    for e in a.entries:
        if e["p"].numel():
            assert _off(e["p"], ref.newton_schulz(e["g"], 5, COEFS, 1e-7)) <= HARD
    b = m.MuonTensors(make())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.moe_lora_muon_step(b, momentum=0.5)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x["p"], y["p"]) and torch.equal(x["m"], y["m"]) for x, y in zip(a.entries, b.entries))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_lora_muon_step(b, momentum=0.5)
    for _ in range(2):
        for gr in grads:
            gr.normal_(generator=g)
        graph.replay()
        m.moe_lora_muon_step(a, momentum=0.5)
        assert all(torch.equal(x["p"], y["p"]) and torch.equal(x["m"], y["m"]) for x, y in zip(a.entries, b.entries))
    m.moe_lora_muon_step(m.MuonTensors([]))
