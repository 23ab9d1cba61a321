"""qmoe_route_backward on routes that were copied, moved or stored in between."""
import numpy as np
import pytest

import f8_util as fu
from gpu_util import qg, to_dev, torch_cuda

pytestmark = pytest.mark.gpu


def _case(T, E, k):
    torch = torch_cuda()
    g = np.random.default_rng([T, E])
    x = to_dev(g.normal(size=(T, E)).astype(np.float32))
    mask = to_dev(g.random(T) >= 0.2)
    return x, mask, to_dev(g.normal(size=(T, k)).astype(np.float32)), torch.full((1,), 0.5, device="cuda")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 24, 4), (300, 65, 3)])
def test_backward_of_a_copied_route(T, E, k):
    q, torch = qg(), torch_cuda()
    x, mask, gw, gl = _case(T, E, k)
    r = q.qmoe_route(x, k, mask=mask)
    want = q.qmoe_route_backward(x, r, grad_weight=gw, grad_loss=gl, mask=mask)
    ref = fu.route(x.double().cpu().numpy(), k, mask.cpu().numpy())
    exact = fu.route_gradient(ref, gw.double().cpu().numpy(), 0.5)
    # weights and p to 2^-18 (the routing's own tests), sums of k and E of them
    size = np.abs(gw.double().cpu().numpy()).max(1, keepdims=True) + 0.5 * E
    fu.assert_close(want.double().cpu().numpy(), exact, 2.0 ** -15 * size + 0 * exact, "dlogits")
    copies = [type(r)(*[t.clone() for t in r]),                                  # each tensor by itself
              type(r)(*[t.cpu().cuda() for t in r]),                             # put away and brought back
              r._replace(tokens=r.tokens.clone()), r._replace(counts=r.counts.clone())]
    for n, c in enumerate(copies):
        d = q.qmoe_route_backward(x, c, grad_weight=gw, grad_loss=gl, mask=mask)
        assert torch.equal(d, want), n


def test_backward_of_a_copied_route_in_a_graph():
    q, torch = qg(), torch_cuda()
    x, mask, gw, gl = _case(200, 16, 2)
    r = q.qmoe_route(x, 2, mask=mask)
    c = type(r)(*[t.clone() for t in r])
    want = q.qmoe_route_backward(x, c, grad_weight=gw, grad_loss=gl, mask=mask)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        d = q.qmoe_route_backward(x, c, grad_weight=gw, grad_loss=gl, mask=mask)
    for turn in range(3):
        gw.mul_(2.0)
        g.replay()
        want = q.qmoe_route_backward(x, r, grad_weight=gw, grad_loss=gl, mask=mask)
        torch.cuda.synchronize()
        assert torch.equal(d, want), turn


def test_routes_of_other_logits_are_refused():
    q, torch = qg(), torch_cuda()
    x, mask, gw, gl = _case(6, 24, 4)
    r = q.qmoe_route(x, 4)
    for bad in (r._replace(counts=r.counts[:23]), r._replace(tokens=r.tokens[:0]), r._replace(weight=r.weight[:5]),
                r._replace(tokens=r.offsets)):
        with pytest.raises(ValueError):
            q.qmoe_route_backward(x, bad, grad_weight=gw)
    for bad in (r._replace(tokens=r.tokens.cpu()), r._replace(counts=r.counts.long())):
        with pytest.raises(TypeError):
            q.qmoe_route_backward(x, bad, grad_weight=gw)
