"""tq_rope inside autograd, as its docstring says: a Function whose backward is the
inverse call, against autograd through the formula in fp64."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
tq = pytest.importorskip("bit_mixed_precision_amd.binding")

from test_decode_gpu import half_ulp  # noqa: E402


class Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, table, pos, interleaved):
        ctx.save_for_backward(table, pos)
        ctx.interleaved = interleaved
        return tq.tq_rope(x, table, pos, interleaved)

    @staticmethod
    def backward(ctx, dy):
        table, pos = ctx.saved_tensors
        return tq.tq_rope(dy.contiguous(), table, pos, ctx.interleaved, True), None, None, None


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_function(dtype, interleaved):
    T, H, D, rot = 37, 5, 96, 64
    dt = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[dtype]
    table = torch.from_numpy(tq.tq_rope_table(100, rot, 1e4, gain=1.25)).cuda()
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(T, H, D, generator=g).to(dt).cuda() for _ in range(2))
    pos = torch.randint(0, 100, (T,), generator=g).int().cuda()
    assert not tq.tq_rope(x.clone().requires_grad_(), table, pos).requires_grad
    x.requires_grad_()
    Rope.apply(x, table, pos, interleaved).backward(dy)

    x64 = x.detach().double().requires_grad_()
    cs = table.double()[pos.long()][:, None]
    cos, sin = cs[..., 0], cs[..., 1]
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else \
        (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x64[..., lo], x64[..., hi]
    y = torch.cat([a * cos - b * sin, b * cos + a * sin, x64[..., rot:]], -1)
    d64 = dy.double()
    y.backward(torch.cat([d64[..., lo], d64[..., hi], d64[..., rot:]], -1))
    want = x64.grad.cpu().numpy()
    # a product and a fused multiply-add in fp32, then one rounding to the type
    mag = torch.zeros_like(d64)
    pair = d64[..., lo].abs() + d64[..., hi].abs()
    mag[..., lo], mag[..., hi] = pair, pair
    before = 2 * 2.0 ** -24 * 1.25 * mag.cpu().numpy()
    err = np.abs(x.grad.double().cpu().numpy() - want)
    assert np.all(err <= before + half_ulp(np.abs(want) + before, dtype))
