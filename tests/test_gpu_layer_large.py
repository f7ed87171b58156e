"""The operators between a layer's products past what one grid or 32 bits of
offset hold."""
import numpy as np
import pytest

from tests import layer_plain as G
from tests import pass_plain as P
from tests.test_gpu_layer import coded, same_codes
from tests.test_gpu_pass import data, dev, host

pytestmark = pytest.mark.gpu


def far_rows(values, dtype, ld):
    """Rows of a host array, ld elements apart on the device."""
    import torch
    t = torch.from_numpy(values).to(P.TYPES[dtype]).cuda()
    wide = torch.empty((values.shape[0] - 1) * ld + values.shape[1], dtype=t.dtype, device="cuda")
    view = wide.as_strided(values.shape, (ld, 1))
    view.copy_(t)
    return view


def test_offsets_past_32_bits():
    """Rows 2^31 elements apart: a row's offset passes 2^32 bytes, and 2^32 elements."""
    import torch
    import optimizer_step_amd as osa
    rows, cols, ld = 4, 300, (1 << 31) + 8
    x, u, dy = (data(s, rows, cols, "bf16") for s in (1, 2, 3))
    far = far_rows(x, "bf16", ld)
    y, q = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"), osa.block_buffers(rows, cols)
    osa.opt_gated_act(far, dev(u, "bf16"), y=y, gate_codes=q)
    want, bound = G.gate(x, u, "silu", "bf16")
    G.check_values(host(y), want, G.stored(want, bound, "bf16"))
    codes, scales = P.encode(x)
    assert np.array_equal(q[0].cpu().numpy()[:, :cols], codes) and np.array_equal(q[1].cpu().numpy()[:, :rows], scales)
    # the backward pass by tiles, its result over the far rows
    dx, t = torch.empty_like(y), osa.block_buffers(cols, rows)
    osa.opt_gated_act_backward(dev(dy, "bf16"), dev(x, "bf16"), dev(u, "bf16"), dgate=dx, dgate_codes_t=t)
    t2 = osa.block_buffers(cols, rows)
    osa.opt_gated_act_backward(dev(dy, "bf16"), far, dev(u, "bf16"), dgate=far, dgate_codes_t=t2)
    assert torch.equal(far, dx) and same_codes(t, t2, cols, rows)
    # a restored matrix
    pair, held = coded(x)
    osa.opt_block_restore(pair, out=far)
    assert np.array_equal(host(far), P.rounded(held, "bf16"))
    # heads of tokens that far apart, in place
    heads = data(5, rows, 256, "bf16")
    far = far_rows(heads, "bf16", ld)
    near = dev(heads, "bf16").view(rows, 2, 128)
    view = far.as_strided((rows, 2, 128), (ld, 128, 1))
    table, out = osa.rotation_table(rows, 128), torch.empty_like(near)
    osa.opt_head_norm(near, None, table=table, q_out=out)
    osa.opt_head_norm(view, None, table=table, q_out=view)
    assert torch.equal(view, out)
    dx = torch.empty_like(near)
    osa.opt_head_norm_backward(out, None, near, None, table=table, dq=dx)
    osa.opt_head_norm_backward(view, None, near, None, table=table, dq=view)
    assert torch.equal(view, dx)


def test_more_tiles_than_a_grid():
    """Rows and columns in more tiles than one launch has workgroups: each takes several in turn."""
    import torch
    import optimizer_step_amd as osa
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for rows, cols in (((1 << 17) + 7, 1025), (3, (1 << 27) + 129)):
        z = torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
        u, dy = z.flip(1).contiguous(), torch.randn(rows, cols, device="cuda", generator=g).bfloat16()
        y, q = torch.empty_like(z), osa.block_buffers(rows, cols)
        osa.opt_gated_act(z, u, y=y, codes=q)
        at = torch.randint(0, rows * cols, (20000,), device="cuda", generator=g)
        at = torch.cat([at, torch.tensor([0, rows * cols - 1], device="cuda")])
        pick = lambda t: t.view(-1)[at]  # noqa: E731
        want, bound = G.gate(host(pick(z)), host(pick(u)), "silu", "bf16")
        G.check_values(host(pick(y)), want, G.stored(want, bound, "bf16"))
        # the transposes: the same as those of each part of 128 * k rows (or columns) alone
        t = osa.block_buffers(cols, rows)
        dup = torch.empty_like(z)
        osa.opt_gated_act_backward(dy, z, u, dup=dup, dup_codes_t=t)
        r, c = (128 * 1000, 1025) if rows > 1000 else (3, 128 * 1000)
        part = osa.block_buffers(cols if rows > 1000 else cols - (1 << 27), rows - r if rows > 1000 else 3)
        cut = (slice(r, None), slice(None)) if rows > 1000 else (slice(None), slice(1 << 27, None))
        osa.opt_gated_act_backward(dy[cut].contiguous(), z[cut].contiguous(), u[cut].contiguous(), dup_codes_t=part)
        if rows > 1000:
            n = rows - r
            assert torch.equal(t[0][:, r:r + n], part[0][:, :n]) and torch.equal(t[1][r // 128:, :cols], part[1][:, :cols])
        else:
            n = cols - (1 << 27)
            assert torch.equal(t[0][1 << 27:, :3], part[0][:, :3]) and torch.equal(t[1][:, 1 << 27:(1 << 27) + n], part[1][:, :n])
        x, t2 = torch.empty_like(z), osa.block_buffers(cols, rows)
        osa.opt_block_restore(q, out=x, codes_t=t2)
        q2 = osa.block_buffers(rows, cols)
        # coded again they stay as they are (a block whose largest value was rounded down to 448 of the next smaller scale takes that one)
        osa.opt_block_cast(x, codes=q2)
        again = torch.empty_like(x)
        osa.opt_block_restore(q2, out=again)
        assert torch.equal(again, x)
        osa.opt_block_cast(x, codes_t=t)
        assert same_codes(t, t2, cols, rows)
        del z, u, dy, y, q, t, dup, part, x, t2, q2, again
        torch.cuda.empty_cache()


def test_more_heads_than_a_grid():
    import torch
    import optimizer_step_amd as osa
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    tokens = (1 << 22) + 5                                  # 2^20 workgroups of four waves, and more
    x = torch.randn(tokens, 1, 64, device="cuda", generator=g).bfloat16()
    k = torch.randn(tokens, 1, 64, device="cuda", generator=g).bfloat16()
    pos = torch.randint(0, 5000, (tokens,), device="cuda", generator=g, dtype=torch.int32)
    table = osa.rotation_table(5000, 64)
    y, z = torch.empty_like(x), torch.empty_like(k)
    dw = torch.empty(64, device="cuda")
    osa.opt_head_norm(x, k, table=table, positions=pos, q_out=y, k_out=z)
    at = torch.cat([torch.randint(0, tokens, (3000,), device="cuda", generator=g), torch.tensor([0, tokens - 1], device="cuda")])
    ones, tab, p = np.ones(64, np.float32), table.cpu().numpy(), pos[at].cpu().numpy()
    for a, b in ((x, y), (k, z)):
        want, bound = G.heads(host(a[at]), ones, tab, p, 1e-6, 64, False)
        G.check_values(host(b[at]), want, G.stored(want, bound, "bf16"))
    dx = torch.empty_like(x)
    osa.opt_head_norm_backward(y, None, x, None, table=table, positions=pos, dq=dx, dweight_q=dw)
    (want, bound), _ = G.head_gradients(host(y[at]), host(x[at]), ones, tab, p, 1e-6, 64, False)
    G.check_values(host(dx[at]), want, G.stored(want, bound, "bf16"))
    # dw in binary64 on the device; a lane adds 128 tokens' heads (4096 waves of 8 slots) in binary32, and 16 more
    r = (x.double().square().mean(-1, keepdim=True) + 1e-6).rsqrt()
    c, s = (v.double()[pos.long()][:, None, :] for v in (table[:, :32], table[:, 32:]))
    a, b = y.double()[..., :32], y.double()[..., 32:]
    dn, m = torch.cat([a * c + b * s, b * c - a * s], -1), torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    want, size = (dn * x.double() * r).sum((0, 1)), (m * x.double().abs() * r).sum((0, 1))
    assert bool(((dw.double() - want).abs() <= (5 + tokens / 4096 + 16) * P.U32 * size).all())
