"""The f8 and routing calls beside autograd: refused where a gradient would be
lost, usable inside a torch.autograd.Function."""
import numpy as np
import pytest

import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda

pytestmark = pytest.mark.gpu


def test_calls_that_would_lose_a_gradient_are_refused():
    q, torch = qg(), torch_cuda()
    N, K, M, E = 32, 128, 4, 8
    W = to_dev(q.qquantize_f8(fu.weights(N, K, seed=1)))
    x = to_dev(fu.acts(M, K, seed=2))
    dy = to_dev(fu.acts(M, N, seed=3)).to(torch.bfloat16)
    logits, gw = torch.randn(M, E, device="cuda"), torch.randn(M, 2, device="cuda")
    xq, r = q.qact_quantize_f8(x), q.qmoe_route(logits, 2)
    one = torch.ones(1, device="cuda")

    def leaf(t):
        return t.detach().clone().requires_grad_()

    calls = [lambda t=leaf(x): q.qact_quantize_f8(t), lambda t=leaf(x): q.qgemv_f8(W, t, N, K),
             lambda t=leaf(dy): q.qgemm_f8_wgrad(t, xq, M, N, K), lambda t=leaf(logits): q.qmoe_route(t, 2),
             lambda t=leaf(gw): q.qmoe_route_backward(logits, r, grad_weight=t),
             lambda t=leaf(one): q.qmoe_route_backward(logits, r, grad_loss=t),
             lambda t=leaf(logits): q.qmoe_route_backward(t, r, grad_weight=gw),
             lambda t=leaf(x): q.qact_quantize_f8(t * 2)]                        # not a leaf
    for n, call in enumerate(calls):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("M,N,K", [(5, 40, 130), (70, 129, 256)])
def test_a_linear_layer_as_a_function(M, N, K):
    """y = f8(x) W^T with both gradients, as a program would write it."""
    q, torch = qg(), torch_cuda()
    w = fu.weights(N, K, seed=1)
    W = to_dev(q.qquantize_f8(w))
    WT = q.qtranspose_f8(W, N, K)

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, master):
            xq = q.qact_quantize_f8(x)
            ctx.save_for_backward(xq)
            return q.qgemm_f8(W, xq, M, N, K)

        @staticmethod
        def backward(ctx, dy):
            xq, = ctx.saved_tensors
            dyb = dy.to(torch.bfloat16)
            return (q.qgemm_f8(WT, q.qact_quantize_f8(dyb), M, K, N), q.qgemm_f8_wgrad(dyb, xq, M, N, K))

    x = to_dev(fu.acts(M, K, seed=2)).requires_grad_()
    master = to_dev(w).requires_grad_()
    g = to_dev(fu.acts(M, N, seed=4))
    (Linear.apply(x, master) * g).sum().backward()
    torch.cuda.synchronize()
    xr = fu.quantize_rows(x.detach().double().cpu().numpy())[0]
    wv = fu.quantize_weights(w)[0]
    dy = g.to(torch.bfloat16).double().cpu().numpy()
    dyr = fu.quantize_rows(dy)[0]
    fu.assert_close(x.grad.double().cpu().numpy(), dyr @ wv, fu.sum_bound(np.abs(dyr) @ np.abs(wv), N), "dx")
    fu.assert_close(master.grad.double().cpu().numpy(), dy.T @ xr, fu.sum_bound(np.abs(dy).T @ np.abs(xr), M), "dw")
