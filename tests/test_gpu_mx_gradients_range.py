"""fp16 gradients of the microscaled layer where one matrix holds groups far below its largest: a
value is exact from 2^-36 of the largest on, and below it off by 2^-40 of the largest at most."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

from trellis_coded_bit_amd import api  # noqa: E402

import mx_check as mc  # noqa: E402
from linear_check import half, tiny  # noqa: E402

F16 = torch.float16


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _spread(g, rows, cols, fmt, far):
    """Groups of columns by turns 1, 2^-far / 2 and 2^-far of the others."""
    e = torch.tensor([0.0, -far / 2, -float(far)], device="cuda")
    s = torch.exp2(e[torch.arange(-(-cols // 32), device="cuda") % 3]).repeat_interleave(32)[:cols]
    return api.mx_pack(_randn(g, rows, cols) * s, fmt)


def _inside(got, a, b, K, lost, what):
    want, mag = a @ b, a.abs() @ b.abs()
    e = mc.gamma(K, F16) * mag + lost
    off, bound = (got.double() - want).abs(), e + half(F16) * (want.abs() + e) + tiny(F16)
    assert bool((off <= bound).all()), f"{what}: {float((off / bound).max()):.3g} of the bound"
    # (far from the type's subnormals, or this would say nothing)
    assert float((want.abs() > 2.0 ** -14).double().mean()) > 0.9


@pytest.mark.parametrize("far", [12, 20, 24])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("B,M,N", [(300, 200, 192), (37, 520, 97), (1000, 64, 300)])
def test_far_groups(B, M, N, fmt, far):
    g = torch.Generator(device="cuda").manual_seed(far)
    w, x = _spread(g, M, N, "fp4", far), _spread(g, B, N, fmt, far)
    W, X = (api.mx_unpack(t, torch.float32).double() for t in (w, x))
    third = (torch.arange(N, device="cuda") // 32) % 3
    # dy such that the groups looked at have gradients that are normal numbers of the type (the
    # largest groups' overflow where the farthest are looked at)
    for c, size in ((third == 2, 8192.0), (third < 2, 2.0 ** (far / 2 - 9))):
        dy = (_randn(g, B, M) * size).clamp(-60000, 60000).to(F16)
        dx, dw, _ = api.mx_linear_backward(dy, w, x)
        d = dy.double()
        lost = [2.0 ** -40 * float(t.abs().max()) * d.abs().sum(i) for t, i in ((W, 1), (X, 0))]
        _inside(dx[:, c], d, W[:, c].contiguous(), M, lost[0][:, None], "dx")
        _inside(dw[:, c], d.t().contiguous(), X[:, c].contiguous(), B, lost[1][:, None], "dw")
