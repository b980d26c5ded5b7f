"""Gradients of the gated linear recurrence on a GB300 against differences of the plain 64-bit one, few entries at
a time."""
import pytest
import torch

import block_testlib as ref
import chunked_gated_delta_gdr_gb300 as gdr

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_gated_delta_gdr_gb300 import build
    build.build()
    if torch.cuda.get_device_capability() != (10, 3):
        pytest.skip("needs sm_103 (GB300)")


def rn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


@pytest.mark.parametrize("name", ["x", "r", "A", "i", "h0"])
@pytest.mark.parametrize("norm", [True, False])
def test_recurrence_gradients_along_few_entries(name, norm):
    # Along directions with four entries of +-1, so that no error hides among thousands of others: a gradient is
    # off by 4 * 2^-22 (n + 16) of its tensor's largest magnitude for n tokens of a segment (all T for A), and
    # four of them by four times that.  Central differences in 64 bits with a step h are off by h^2 times a
    # third derivative and by 2^-53 of the loss's terms over h; with h = 1e-5 below 1e-7 of the largest
    # gradient.
    T, cu = ref.CU["ghosts"]
    D, n = 24, len(cu) - 1
    cud = torch.tensor(cu, dtype=torch.int32, device=DEV)
    s = dict(x=rn(1, T, D), r=rn(2, T, D), i=rn(3, T, D), h0=rn(4, n, D), dy=rn(5, T, D), dht=rn(6, n, D),
             A=8 * torch.log(0.9 + 0.099 * torch.rand(D, generator=torch.Generator().manual_seed(7))))
    d = {k: v.to(DEV) for k, v in s.items()}
    grads = dict(zip(("x", "r", "A", "i", "h0"), gdr.rec_bwd(d["x"], d["r"], d["A"], d["dy"], d["i"], norm, d["h0"],
                                                             cud, d["dht"])))
    base = {k: s[k].double() for k in grads}

    def loss(v):
        y, h, _ = ref.rec(v["x"], v["r"], v["A"], v["i"], norm, v["h0"], cu)
        return float((y * s["dy"].double()).sum() + (h * s["dht"].double()).sum())

    g = grads[name].cpu().double()
    long = max(e - b for b, e in zip(cu, cu[1:]))
    tol = 4 * 4 * 2.0 ** -22 * ((T if name == "A" else long) + 16) * float(g.abs().max())
    # the directions tell a gradient from one that is 5 % off
    gen = torch.Generator().manual_seed(8)
    sizes = []
    for _ in range(6):
        way = torch.zeros(g.numel(), dtype=torch.float64)
        at = torch.randperm(g.numel(), generator=gen)[:4]
        way[at] = 2.0 * torch.randint(0, 2, (4,), generator=gen).double() - 1
        way, h = way.view(g.shape), 1e-5
        diff = (loss({**base, name: base[name] + h * way}) - loss({**base, name: base[name] - h * way})) / (2 * h)
        sizes.append(abs(diff))
        assert abs(float((g * way).sum()) - diff) <= tol + 1e-7 * float(g.abs().max()), name
    assert max(sizes) * 0.05 > tol + 1e-7 * float(g.abs().max())
