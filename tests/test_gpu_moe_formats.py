"""The operators around the experts run together, as the example runs them: 8-bit and BF16 layers, and the
gradients of a BF16 layer."""
import pytest
import torch

from examples import moe_layer
from tp_reduce_residual_gb300 import beamnorm as bn
from tp_reduce_residual_gb300 import build as nbuild

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "the GPU tests need a CUDA device"
    nbuild.build()
    bn.load()
    bn.check_device_error(raise_on_error=False)
    yield
    assert bn.check_device_error() == 0


# activations rounded three times: to half a code of 127 (about 2^-7 of a row's largest value, 2^-5 of a typical
# one, and sums average it down), or to BF16's 2^-8
@pytest.mark.parametrize("fmt,most", [("int8", 0.05), ("bf16", 0.02)])
def test_layer_runs(fmt, most):
    assert moe_layer.main(["--format", fmt, "--tokens", "37", "--hidden", "512", "--width", "256"]) < most
    assert moe_layer.main(["--format", fmt, "--tokens", "3", "--hidden", "256", "--width", "128", "--shards", "1", "--experts", "6",
                           "--topk", "2"]) < most


@pytest.mark.parametrize("T,H,F,E,k,R", [(23, 256, 128, 6, 2, 2), (70, 512, 256, 16, 4, 1), (1, 128, 64, 4, 1, 1)])
def test_gradients_against_the_formulas(T, H, F, E, k, R):
    """Against 64-bit automatic differentiation of elementary operations, with the same experts and weights.  Each
    gradient passes up to five roundings to BF16 of 2^-8 that vary in sign: 2^-6 of its norm."""
    layer = moe_layer.MoELayer(H, F, E, k, R, "bf16")
    g = torch.Generator(device="cuda").manual_seed(T)
    h = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dz = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    got = layer.gradients(h, dz)
    ids, w = layer.route(h.float() @ layer.router.T)
    leaves = dict(h=h.double().requires_grad_(), w=w.double().requires_grad_())
    up = [u.double().requires_grad_() for u in layer.up]
    down = [d.double().requires_grad_() for d in layer.down]
    (layer.mixture(leaves["h"], up, down, ids, leaves["w"]) * dz.double()).sum().backward()
    for name, mine, want in [("h", got["h"], leaves["h"].grad), ("w", got["w"], leaves["w"].grad)] \
            + [(f"up{r}", got["up"][r], up[r].grad) for r in range(R)] + [(f"down{r}", got["down"][r], down[r].grad) for r in range(R)]:
        assert mine.shape == want.shape and float((mine.double() - want).norm() / want.norm()) < 2.0 ** -6, name


def test_gradients_against_differences():
    """The layer's own change along the gradient of one expert's weights and of the rows."""
    layer = moe_layer.MoELayer(256, 128, 4, 2, 1, "bf16")
    g = torch.Generator(device="cuda").manual_seed(9)
    h = torch.randn(40, 256, generator=g, device="cuda").bfloat16()
    dz = torch.randn(40, 256, generator=g, device="cuda").bfloat16()
    ids, w = layer.route(h.float() @ layer.router.T)
    got = layer.gradients(h, dz)
    up, down = [u.double() for u in layer.up], [d.double() for d in layer.down]

    def value(h, up, down):
        return (layer.mixture(h, up, down, ids, w.double()) * dz.double()).sum()

    step = 2.0 ** -10
    for which in ("up", "down", "h"):
        v = got[which] if which == "h" else got[which][0]
        v = v.double() / v.double().norm()
        ends = [value(h.double() + s * v, up, down) if which == "h" else
                value(h.double(), [up[0] + s * v], down) if which == "up" else value(h.double(), up, [down[0] + s * v]) for s in (step, -step)]
        slope = (ends[0] - ends[1]) / (2 * step)
        want = ((got[which] if which == "h" else got[which][0]).double() * v).sum()
        # second differences vanish to step^2; the gradient itself is within 2^-6
        assert abs(slope - want) <= 2.0 ** -6 * abs(want) + 1e-3, (which, float(slope), float(want))


def test_two_calls_and_a_graph():
    """A captured layer, replayed on other inputs while the same layer runs eagerly, gives the eager results."""
    for fmt in ("int8", "bf16"):
        layer = moe_layer.MoELayer(256, 128, 8, 2, 2, fmt)
        g = torch.Generator(device="cuda").manual_seed(2)
        h, residual = (torch.randn(50, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
        fixed_h, fixed_r = h.clone(), residual.clone()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            layer(fixed_h, fixed_r.clone())
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = fixed_r.clone()
            out = layer(fixed_h, res)
        for i in range(3):
            new = torch.randn(50, 256, generator=g, device="cuda").bfloat16()
            fixed_h.copy_(new)
            graph.replay()
            eager_res = residual.clone()
            eager = layer(new, eager_res)
            torch.cuda.synchronize()
            assert torch.equal(out, eager) and torch.equal(res, eager_res), (fmt, i)
