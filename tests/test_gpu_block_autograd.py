"""The operators around the experts beside torch's autograd: what they write counts as changed in place, and they
serve as the two halves of a torch.autograd.Function."""
import pytest
import torch

import block_ref as ref
import harness

pytestmark = pytest.mark.gpu
bf = torch.bfloat16


def rand(*s, dtype=bf):
    return torch.randn(*s, device="cuda").to(dtype)


def saved_then(write, *shape, dtype=bf):
    """A tensor that autograd saves for a square's gradient, and which `write` then fills."""
    leaf = rand(*shape, dtype=dtype).requires_grad_()
    t = leaf * 1
    loss = (t * t).sum()
    with torch.no_grad():
        write(t)
    with pytest.raises(RuntimeError, match="inplace operation"):
        loss.backward()


def test_a_saved_tensor_that_is_written_raises_in_the_backward_pass():
    import fp4_expert_gemv_b200 as fe
    x, w, r, h, l = rand(4, 64), rand(32, 64), rand(4, 64), rand(64), rand(4, 8, dtype=torch.float32)
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    _, counts, n = fe.balance_loss(l, idx)
    saved_then(lambda t: fe.linear(x, w, y=t), 4, 32)
    saved_then(lambda t: fe.linear(x, w, z=t), 4, 32)
    saved_then(lambda t: fe.linear(x, w, residual=t, y=t), 4, 32)
    saved_then(lambda t: fe.linear(x, w, y=t, stream=torch.cuda.current_stream()), 4, 32)
    saved_then(lambda t: fe.block_norm(r, x, r_out=t), 4, 64)
    saved_then(lambda t: fe.block_norm(t, x, r_out=t), 4, 64)
    saved_then(lambda t: fe.block_norm(r, w_pre=h, u=t), 4, 64)
    saved_then(lambda t: fe.balance_loss(l, idx, loss=t), 3, dtype=torch.float32)
    saved_then(lambda t: fe.balance_loss_backward(l, counts, n, 2, dlogits=t), 4, 8)
    gl = harness.GpuLayer(8, 256, 128, 0, max_T=4, max_k=2)
    R, wr, H = rand(3, 256), rand(8, 256), rand(256)
    saved_then(lambda t: gl.layer.forward_block(R, 2, wr, w_pre=H, r_out=t), 3, 256)
    saved_then(lambda t: gl.layer.forward_block(R, 2, wr, w_pre=H, w_next_pre=H, u_out=t), 3, 256)
    saved_then(lambda t: gl.layer.forward_block(R, 2, wr, w_pre=H, logits=t), 3, 8, dtype=torch.float32)
    with pytest.raises(ValueError, match="requires grad"):
        gl.layer.forward_block(R, 2, wr.clone().requires_grad_(), w_pre=H)
    gl.layer.close()
    torch.cuda.synchronize()


def test_as_an_autograd_function():
    """gelu(x w^T + b) with the pair of calls: the gradients that autograd finds are linear_backward's, bit by bit,
    and those of the formula (dz rounded to bf16: half a step of each factor)."""
    import fp4_expert_gemv_b200 as fe

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            z = x.new_empty(x.shape[0], w.shape[0])
            y = fe.linear(x, w, bias=b, act=fe.ACT_GELU, z=z)
            ctx.save_for_backward(x, w, z)
            return y

        @staticmethod
        def backward(ctx, dy):
            x, w, z = ctx.saved_tensors
            dx, dw, db = fe.linear_backward(dy.contiguous(), x, w, z=z, act=fe.ACT_GELU)
            return dx, dw, db.to(bf)

    x, w, b = rand(50, 64).requires_grad_(), (rand(32, 64).float() / 8).to(bf).requires_grad_(), rand(32).requires_grad_()
    dy = rand(50, 32)
    y = Linear.apply(x, w, b)
    y.backward(dy)
    with torch.no_grad():
        z = torch.empty(50, 32, dtype=bf, device="cuda")
        assert torch.equal(fe.linear(x, w, bias=b, act=fe.ACT_GELU, z=z), y)
        dx, dw, db = fe.linear_backward(dy, x, w, z=z, act=fe.ACT_GELU)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw) and torch.equal(b.grad, db.to(bf))
    dz, mag = ref.linear_dz(dy, z, "gelu")
    edz = 2.0 ** -8 * dz.abs() + ref.FWD * mag
    W = w.detach().double()
    ref.close(x.grad, dz @ W, edz @ W.abs() + (32 / 16 + 4) * 2.0 ** -22 * ((dz.abs() + edz) @ W.abs()), "dx")
