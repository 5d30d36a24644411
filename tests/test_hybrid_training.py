"""The hybrid stack with linear attention: prompt and steps, and training over packed documents with its gradients."""
import pytest
import torch

from delta_rule_recurrent_gated_gb300 import binding, hybrid

pytestmark = pytest.mark.gpu


def test_prompt_and_steps_of_linear_attention_agree_with_the_whole():
    B, T, steps, hidden = 2, 150, 5, 256
    x = torch.randn(B, T + steps, hidden, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    whole = hybrid.HybridStack(B, linear="decay")(x)
    stack = hybrid.HybridStack(B, linear="decay")
    got = torch.cat([stack(x[:, :T])] + [stack(x[:, T + i:T + i + 1]) for i in range(steps)], 1)
    assert stack.status() == binding.DR_OK and got.isfinite().all()
    rel = lambda a, b: float((a - b).float().norm() / b.float().norm())  # noqa: E731
    # the bounds of the delta-rule stack (test_hybrid.py): bf16 activations through four layers, codes of 2^-7
    assert rel(got[:, :T], whole[:, :T]) < 2e-2 and rel(got[:, T:], whole[:, T:]) < 4e-2


def test_a_step_in_a_captured_graph():
    B, hidden = 2, 256
    xs = torch.randn(5, B, 1, hidden, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    plain, graphed = (hybrid.HybridStack(B, linear="decay") for _ in range(2))
    prompt = torch.randn(B, 70, hidden, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    plain(prompt), graphed(prompt)
    x = xs[0].clone()
    plain(xs[0]), graphed(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = graphed(x)
    for i in range(1, 5):
        ref = plain(xs[i])
        x.copy_(xs[i])
        g.replay()
        assert torch.equal(y, ref)


def plain_stack(stack, x, lens):
    """The same layers as torch operations in 64 bits, for autograd; returns y and the weights by layer."""
    weights = []
    leaf = lambda t: t.detach().double().cpu().requires_grad_()  # noqa: E731
    for layer in stack.layers:
        w = {n: leaf(getattr(layer, n)) for n in ("w_in", "w_out", "wq", "wk") if hasattr(layer, n)}
        weights.append(w)
        d, outs = layer.d, []
        qkv = (x @ w["w_in"]).reshape(x.shape[0], -1, d)
        for part in qkv.split(lens):
            n = part.shape[0]
            back = torch.arange(n)[:, None] - torch.arange(n)
            if "wq" in w:
                q, k, v = part.split(layer.heads, 1)
                norm = lambda t, s: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * s  # noqa: E731
                cos, sin = (t.double().cpu()[:n, None] for t in (layer.cos, layer.sin))

                def turn(t):
                    a, b = t.chunk(2, -1)
                    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

                q, k = turn(norm(q, w["wq"])), turn(norm(k, w["wk"]))
                G = q.shape[1] // k.shape[1]
                k, v = (t.repeat_interleave(G, 1) for t in (k, v))
                s = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
                p = s.masked_fill(back < 0, -float("inf")).softmax(-1)
            else:
                q, k, v = part.split(layer.H, 1)
                g = layer.g.double().cpu()[:, None, None]
                p = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5 * torch.exp(g * back.clamp(min=0)) * (back >= 0)
            outs.append(torch.einsum("hij,jhd->ihd", p, v).flatten(1))
        x = x + torch.cat(outs) @ w["w_out"]
    return x, weights


@pytest.mark.parametrize("io,bound", [("f32", 2e-4), ("bf16", 6e-2)])
def test_training_over_packed_documents(io, bound):
    """Gradients of every weight and of the input against autograd of the same stack in 64 bits, relative to their
    norms.  bf16: each of the four layers rounds about six tensors on the way and six on the way back, each by 2^-9 of
    its norm at a guess of random signs and by 2^-8 at most: 48 2^-9 / sqrt(48) = 1.4e-2 is expected and four times that
    is the bound.  fp32: the same count at 2^-24 and the sums over up to 260 tokens and 512 channels, 2^-15 together,
    with the same factor and room for torch's own products: 2e-4."""
    lens = [130, 0, 1, 260, 57]
    tokens = sum(lens)
    gen = torch.Generator().manual_seed(5)
    kind = torch.bfloat16 if io == "bf16" else torch.float32
    x, dy = (torch.randn(tokens, 256, generator=gen).to(kind) for _ in range(2))
    cu = torch.tensor([0, 130, 130, 131, 391, 448], dtype=torch.int32).cuda()
    stack = hybrid.TrainingStack(tokens, len(lens), io=io)
    y = stack.forward(x.cuda(), cu)
    dx = stack.backward(dy.cuda())
    x64 = x.double().requires_grad_()
    y64, weights = plain_stack(stack, x64, lens)
    (y64 * dy.double()).sum().backward()
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    errors = {"y": rel(y, y64.detach()), "dx": rel(dx, x64.grad)}
    for i, (layer, w) in enumerate(zip(stack.layers, weights)):
        assert set(layer.grads) == set(w)
        errors |= {f"{i}.{n}": rel(layer.grads[n], w[n].grad) for n in w}
    assert all(e < bound for e in errors.values()), errors


def test_training_step_in_a_captured_graph():
    """One graph of forward and backward takes other documents of the same rows."""
    tokens, lens = 300, [[100, 150, 50], [300, 0, 0]]
    gen = torch.Generator().manual_seed(6)
    x, dy = (torch.randn(tokens, 256, generator=gen).bfloat16().cuda() for _ in range(2))
    cus = [torch.tensor([0, a, a + b, a + b + c], dtype=torch.int32).cuda() for a, b, c in lens]
    stack, cu = hybrid.TrainingStack(tokens, 3), cus[0].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        stack.forward(x, cu), stack.backward(dy)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = stack.forward(x, cu)
            dx = stack.backward(dy)
            grads = [layer.grads for layer in stack.layers]
    torch.cuda.synchronize()
    other = hybrid.TrainingStack(tokens, 3)
    for c in cus:
        cu.copy_(c)
        graph.replay()
        want = other.forward(x, c), other.backward(dy)
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dx, want[1])
        assert all(torch.equal(a[n], layer.grads[n]) for a, layer in zip(grads, other.layers) for n in a)
