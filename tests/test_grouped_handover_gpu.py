"""What the two CTAs of a pair hand each other in the grouped products: rows
that one of them has gathered are read by MMAs that the other issues.  Calls
follow each other on inputs in turn, so that a row read too early would be the
other input's, and every call has to give the same bits as the first."""
import pytest
import torch

import swiglu_mlp_projection_gb300 as swg

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF = torch.bfloat16


@pytest.mark.parametrize("T,E,k,d,d_ff", [(1, 8, 2, 4096, 1024), (40, 8, 2, 2048, 512),
                                          (700, 4, 2, 1032, 264), (4096, 16, 2, 512, 256)])
def test_stages_of_two_inputs_in_turn(cuda_lib, T, E, k, d, d_ff):
    g = torch.Generator(device=DEV).manual_seed(T)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)
    xs = [normal(T, d) for _ in range(3)]
    wg, wu = normal(E, d, d_ff, scale=d ** -0.5), normal(E, d, d_ff, scale=d ** -0.5)
    rt = [swg.route(torch.randn(T, E, generator=g, device=DEV), k) for _ in xs]
    want = []
    for x, r in zip(xs, rt):
        h = swg.experts_up(x, wg, wu, r)
        # (the first results against the definition in 64 bits)
        e = torch.bucketize(torch.arange(T * k, device=DEV), r.offsets[1:].long(), right=True)
        for row in range(0, T * k, max(1, T * k // 16)):
            a = x[r.order[row].long() // k].double()
            gg, uu = a @ wg[e[row]].double(), a @ wu[e[row]].double()
            ref = gg * torch.sigmoid(gg) * uu
            tol = 2.0 ** -8 * ref.abs() + 64 * d ** 0.5 * 2.0 ** -24
            assert bool(((h[row].double() - ref).abs() <= tol).all())
        want.append(h)
    out = torch.empty_like(want[0])
    for rep in range(60):
        i = rep % 3
        swg.experts_up(xs[i], wg, wu, rt[i], out=out)
        assert torch.equal(out, want[i]), rep
    swg.check_device_status()
