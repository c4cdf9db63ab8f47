"""Products with NVFP4 weights whose weight, scales, global scale and bias the kernels
launched just before them write, each programmatically, with nothing between them: what
a call reads ahead of its grid-dependency wait would be the call's before.
"""
import pytest
import torch

from .test_linear_nvfp4_gpu import BF, DEV, F32, gen, mbx, rnd  # noqa: F401

pytestmark = pytest.mark.gpu


# the digits made beforehand and by the product; one slice of K and several; rows copied by TMA and by warps
@pytest.mark.parametrize("rows,N,K", [(16, 10006, 2048), (16, 5000, 5120), (40, 3000, 4096), (2, 5000, 5120), (16, 6000, 1040),
                                      (1, 700, 1024)])
def test_a_weight_written_directly_before(mbx, rows, N, K):  # noqa: F811
    g = gen(N)
    ms = [rnd(g, (N, K), BF) for _ in range(3)]
    sc, sh, x = rnd(g, (1, K), BF, 0.1), rnd(g, (1, K), BF, 0.1), rnd(g, (rows, K), BF)
    # bias = r + gate * u; the global scale is an element of a modulation table
    rs, gate, u = [rnd(g, (2, N // 2), BF) for _ in range(3)], rnd(g, (1, N // 2), BF), rnd(g, (2, N // 2), BF)
    table, tembs = torch.full((1, 6, 8), 300.0, device=DEV), [torch.full((1, 48), 50.0 * i, device=DEV) for i in range(3)]
    normed = torch.empty((N, K), dtype=BF, device=DEV)
    q4, sf = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV), torch.zeros(mbx.nvfp4_sf_shape(N, K), dtype=torch.uint8, device=DEV)
    bias, planes = torch.zeros((2, N // 2), dtype=BF, device=DEV), torch.zeros((6, 1, 8), device=DEV)
    gs = planes.view(-1)[:1]

    def call(i, order, sync):
        write = [lambda: mbx.ln_modulate_nvfp4(ms[i], sc, sh, gs, variant="high", out=normed, out_fp4=q4, out_sf=sf),
                 lambda: mbx.residual_gate_add(rs[i], gate, u, variant="high", out=bias)]
        mbx.modulation_table_add(table, tembs[i], out=planes)
        for w in write[::order]:
            w()
            if sync:
                torch.cuda.synchronize()
        return mbx.linear_nvfp4(x, q4, sf, gs, bias.view(-1), True)

    want = [call(i, 1, True) for i in range(3)]
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1]) and not torch.equal(want[1], want[2])
    got = [(i, call(i, order, False)) for _ in range(10) for order in (1, -1) for i in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in got)


@pytest.mark.parametrize("rows,N,K", [(16, 10007, 2048), (16, 5000, 5120), (2, 5000, 5120), (1, 700, 1024)])
def test_a_global_scale_written_directly_before(mbx, rows, N, K):  # noqa: F811
    g = gen(N + 1)
    w4, sf, gs0 = mbx.nvfp4_weight(rnd(g, (N, K), BF, 0.03))
    x = rnd(g, (rows, K), BF)
    table, tembs = gs0.reshape(1, 1, 1).expand(1, 6, 8).contiguous(), [torch.full((1, 48), 700.0 * i, device=DEV) for i in range(3)]
    planes = torch.zeros((6, 1, 8), device=DEV)

    def call(i, sync):
        mbx.modulation_table_add(table, tembs[i], out=planes)
        if sync:
            torch.cuda.synchronize()
        return mbx.linear_nvfp4(x, w4, sf, planes.view(-1)[:1])

    want = [call(i, True) for i in range(3)]
    got = [(i, call(i, False)) for _ in range(30) for i in range(3)]
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    assert all(torch.equal(o, want[i]) for i, o in got)
