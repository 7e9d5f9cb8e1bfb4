"""A pre-norm gated feed-forward block trained with 8-bit saved activations.

    y = x + W2 swiglu(W1 layer_norm(x))

for bf16 x (T, D), W1 (2F, D), W2 (D, F), T, D and F multiples of 32.  Every
product runs on the block-scaled tensor cores on MX casts of its operands, and
everything that the backward pass needs of the forward pass is kept as MX bytes:

    what is kept                                            bytes a token
    the norm's input, from layer_norm(save=True)            33/32 D
    the norm's output, its dim1 cast (for dW1)              33/32 D
    the activation's input, from swiglu(save=True)          33/32 2F
    the activation's output, its dim1 cast (for dW2)        33/32 F
    the norm's statistics                                   8

half of what bf16 would take (4 D + 6 F).  The operators' results carry no graph, so
the block can be differentiated once; a second derivative raises an error.  Run as a
program, it trains the block for a few steps on the current GPU and prints the loss
and the bytes kept.
"""
import torch

import mxfp8_block_scaled_dim0_gb300 as mx


def _dense(t):
    """t, or a copy of it where the operators could not read it in place: rows
    apart, transposed, or off the 16-byte boundary."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() % 16 else t


class _Once(torch.autograd.Function):
    """Its inputs but the first, as results that cannot be differentiated."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return tuple(g.view_as(g) for g in grads)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("FeedForward has no second derivative")


class _Block(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, norm_w, norm_b, w1, w2, eps):
        n, mean, rstd, xq, xs = mx.layer_norm(x, norm_w, norm_b, eps, save=True)
        n0, ns0, n1, ns1 = mx.cast_dim0_dim1(n)
        a0, as0, a1, as1 = mx.cast_dim0_dim1(w1)
        h, gq, gs = mx.swiglu(mx.matmul(n0, ns0, a0, as0), save=True)
        h0, hs0, h1, hs1 = mx.cast_dim0_dim1(h)
        b0, bs0, b1, bs1 = mx.cast_dim0_dim1(w2)
        y = mx.matmul(h0, hs0, b0, bs0)
        # a1 and b1 are of the weights, not of the batch: kept as they are.
        ctx.save_for_backward(xq, xs, mean, rstd, n1, ns1, gq, gs, h1, hs1, norm_w, a1, as1, b1, bs1)
        return x + y

    @staticmethod
    def backward(ctx, dy):
        with torch.no_grad():
            grads = _Block.gradients(dy, *ctx.saved_tensors)
        if torch.is_grad_enabled():
            # create_graph=True.  The gradients depend on x and the weights even where
            # dy is a constant: the anchor, not dy, brings them into the graph.
            grads = _Once.apply(torch.empty(0, requires_grad=True), *grads)
        return (*grads, None)

    @staticmethod
    def gradients(dy, xq, xs, mean, rstd, n1, ns1, gq, gs, h1, hs1, norm_w, a1, as1, b1, bs1):
        dy = _dense(dy)
        d0, ds0, d1, ds1 = mx.cast_dim0_dim1(dy)
        dw2 = mx.matmul(d1, ds1, h1, hs1)
        dgu = mx.swiglu_backward(mx.matmul(d0, ds0, b1, bs1), (gq, gs))
        e0, es0, e1, es1 = mx.cast_dim0_dim1(dgu)
        dw1 = mx.matmul(e1, es1, n1, ns1)
        dn = mx.matmul(e0, es0, a1, as1)
        dx, dw, db = mx.layer_norm_backward(dn, (xq, xs), norm_w, mean, rstd)
        return dy + dx, dw, db, dw1, dw2


class FeedForward(torch.nn.Module):
    """The block.  Norm parameters in float32, weights in bf16."""

    def __init__(self, dim, hidden, eps=1e-5, device="cuda"):
        super().__init__()
        if dim % 32 or hidden % 32:
            raise ValueError("dim and hidden must be multiples of 32, got %d and %d" % (dim, hidden))
        self.eps = eps
        self.norm_w = torch.nn.Parameter(torch.ones(dim, device=device))
        self.norm_b = torch.nn.Parameter(torch.zeros(dim, device=device))
        self.w1 = torch.nn.Parameter(torch.randn(2 * hidden, dim, device=device)
                                     .mul_(dim ** -0.5).to(torch.bfloat16))
        self.w2 = torch.nn.Parameter(torch.randn(dim, hidden, device=device)
                                     .mul_(hidden ** -0.5).to(torch.bfloat16))

    def forward(self, x):
        shape = x.shape
        x = x.reshape(-1, shape[-1])
        if x.shape[0] % 32:
            raise ValueError("the number of tokens must be a multiple of 32, got %d" % x.shape[0])
        return _Block.apply(_dense(x), self.norm_w, self.norm_b, self.w1, self.w2, self.eps).reshape(shape)


def main(tokens=4096, dim=1024, hidden=4096, steps=5):
    torch.manual_seed(0)
    block = FeedForward(dim, hidden)
    x = torch.randn(tokens, dim, device="cuda").to(torch.bfloat16)
    target = torch.randn(tokens, dim, device="cuda").to(torch.bfloat16)
    opt = torch.optim.SGD(block.parameters(), lr=0.5)
    kept = 33 * tokens * (2 * dim + 3 * hidden) // 32 + 8 * tokens
    print("kept for the backward pass: %.1f MB (bf16: %.1f MB)"
          % (kept / 1e6, tokens * (4 * dim + 6 * hidden) / 1e6))
    for step in range(steps):
        loss = (block(x).float() - target.float()).square().mean()
        opt.zero_grad(set_to_none=True)
        loss.backward()
        opt.step()
        print("step %d  loss %.4f" % (step, loss.item()))


if __name__ == "__main__":
    main()
