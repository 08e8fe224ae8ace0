"""The bf16 / fp16 operators beside other autograd nodes: given outputs are in-place writes that autograd
notices, and what the backward needs is saved where torch's saved-tensor hooks see it."""
import pytest
import torch

import nvfp4_block_scaled_mxfp8_amd as g
from mm_util import randn

pytestmark = pytest.mark.gpu

M, N, K, G, R, T, k, E = 48, 64, 64, 3, 8, 24, 2, 4
BF = torch.bfloat16


def _writes():
    """(name, a given output, a call that writes it)."""
    x, w, dy = randn((M, K), BF, 1).cuda(), randn((G, N, K), BF, 2).cuda(), randn((M, N), BF, 3).cuda()
    m = torch.tensor([20, 0, 28], dtype=torch.int32, device="cuda")
    a, b = randn((2, R, K), BF, 4).cuda(), randn((2, N, R), BF, 5).cuda()
    ids = (torch.arange(M, device="cuda") % 3 - 1).to(torch.int32)
    plan = g.dispatch_plan((torch.arange(T * k, device="cuda") % E).to(torch.int32).view(T, k), E)
    tok, row = randn((T, K), BF, 6).cuda(), randn((T * k, K), BF, 7).cuda()

    def new(*shape, dtype=BF):
        return torch.ones(shape, dtype=dtype, device="cuda")
    for name, out, call in (
            ("forward", new(M, N), lambda o: g.grouped_matmul_forward(x, w, m, out=o)),
            ("dgrad", new(M, K), lambda o: g.grouped_matmul_dgrad(dy, w, m, out=o)),
            ("wgrad", new(G, N, K), lambda o: g.grouped_matmul_wgrad(dy, x, m, out=o)),
            ("wgrad fp32", new(G, N, K, dtype=torch.float32), lambda o: g.grouped_matmul_wgrad(dy, x, m, g.OUT_FP32, out=o)),
            ("wgrad added", new(G, N, K, dtype=torch.float32),
             lambda o: g.grouped_matmul_wgrad(dy, x, m, g.OUT_FP32_ACCUMULATE, out=o)),
            ("dispatch", new(T * k, K), lambda o: g.dispatch_forward(tok, plan, out=o)),
            ("combine", new(T, K), lambda o: g.combine_forward(row, plan, out=o)),
            ("dispatch gradient", new(T, K), lambda o: g.dispatch_backward(row, plan, out=o)),
            ("adapters", new(M, N), lambda o: g.lora_forward(dy, x, a, b, ids, out=o)),
            ("adapters in place", new(M, N), lambda o: g.lora_forward(o, x, a, b, ids, out=o))):
        yield name, out, call


def test_a_given_output_that_autograd_saved_is_noticed():
    """A node saved the tensor before it was written: its backward raises, as for a torch in-place operation."""
    for name, out, call in _writes():
        print(f"given output: {name}", flush=True)
        leaf = torch.ones_like(out).requires_grad_()
        y = leaf * out                                    # saves out for leaf's gradient
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_an_accumulated_main_grad_that_autograd_saved_is_noticed():
    x, w, dy = randn((M, K), BF, 1).cuda(), randn((G, N, K), BF, 2).cuda().requires_grad_(), randn((M, N), BF, 3).cuda()
    m = torch.tensor([20, 0, 28], dtype=torch.int32, device="cuda")
    w.main_grad = torch.zeros(w.shape, device="cuda")
    leaf = torch.ones_like(w.main_grad).requires_grad_()
    y = leaf * w.main_grad
    g.grouped_matmul(x, w, m, accumulate_main_grad=True).backward(dy)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_inputs_and_new_outputs_are_not_touched():
    x, w = randn((M, K), BF, 1).cuda(), randn((G, N, K), BF, 2).cuda()
    m = torch.tensor([20, 0, 28], dtype=torch.int32, device="cuda")
    y = g.grouped_matmul_forward(x, w, m)
    assert [t._version for t in (x, w, m, y)] == [0, 0, 0, 0]
    with torch.inference_mode():
        out = torch.empty_like(y)
        g.grouped_matmul_forward(x, w, m, out=out)
    assert torch.equal(out, y)


def test_the_adapters_context_passes_the_saved_tensor_hooks():
    """Everything that lora's backward reads goes through the hooks (offloading to the host, say), gives the
    same bits after a round trip, and is let go with the graph."""
    t = [randn((M, N), BF, 1).cuda(), randn((M, K), BF, 2).cuda(), randn((2, R, K), BF, 3).cuda(), randn((2, N, R), BF, 4).cuda()]
    ids = (torch.arange(M, device="cuda") % 3 - 1).to(torch.int32)
    wide = torch.tensor([0.5, 9.0, 1.5, 9.0], device="cuda")
    dy = randn((M, N), BF, 5).cuda()
    for scales in (None, torch.tensor([0.5, 1.5], device="cuda"), wide[::2]):
        grads, seen = [], []

        def pack(s):
            seen.append(s.nbytes)
            return s.cpu()
        for hooks in (False, True):
            leaf = [v.clone().requires_grad_() for v in t]
            if hooks:
                with torch.autograd.graph.saved_tensors_hooks(pack, lambda s: s.cuda()):
                    y = g.lora(*leaf, ids, scales)
            else:
                y = g.lora(*leaf, ids, scales)
            y.backward(dy)
            grads.append([v.grad for v in leaf])
        assert all(torch.equal(p, q) for p, q in zip(*grads))
        assert sum(seen) >= sum(v.nbytes for v in t[1:]) + g.lora_query_sizes(M, K, N, R, 2)["ctx_bytes"]
