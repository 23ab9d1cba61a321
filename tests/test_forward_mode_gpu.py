"""The f8, routing and attention calls beside forward-mode differentiation: refused where a tangent would be lost,
usable inside functions that say how theirs goes on."""
import pytest

from gpu_util import qg, torch_cuda

pytestmark = pytest.mark.gpu


def test_calls_that_would_lose_a_tangent_are_refused():
    q, torch = qg(), torch_cuda()
    fw = torch.autograd.forward_ad
    bf = torch.bfloat16
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    x = torch.randn(2, 4, 128, device="cuda", dtype=bf)
    rows = torch.randn(2, 128, device="cuda")
    f, g = torch.rand(64, device="cuda"), torch.ones(128, device="cuda")
    cache = q.qkv_cache(2, 16, 4, 128)
    packed = torch.zeros(q.qpacked_bytes_f8(64, 128), dtype=torch.uint8, device="cuda")
    xq = q.qact_quantize_f8(rows)
    route = q.qmoe_route(rows[:, :8].contiguous(), 2)
    dy = torch.randn(2, 64, device="cuda", dtype=bf)

    def dual(t):
        return fw.make_dual(t, torch.ones_like(t))

    calls = [lambda d: q.qhead_norm_rope(d(x), x, pos, f), lambda d: q.qhead_norm_rope(x, d(x), pos, f),
             lambda d: q.qhead_norm_rope(x, d(x)[:, :2], pos, f),
             lambda d: q.qhead_norm_rope(x, x, pos, f, d(g), g), lambda d: q.qhead_norm_rope(x, x, pos, f, g, d(g)),
             lambda d: q.qhead_norm_rope(x, x, pos, d(f)),
             lambda d: q.qhead_norm_rope_backward(d(x), x, x, x, pos, f),
             lambda d: q.qkv_write(cache, d(x), x, pos), lambda d: q.qkv_write(cache, x, d(x), pos),
             lambda d: q.qkv_norm_rope_write(cache, x, x, d(x), pos, pos, f),
             lambda d: q.qattn_decode(cache, d(x), table, pos),
             lambda d: q.qact_quantize_f8(d(rows)), lambda d: q.qgemv_f8(packed, d(rows), 64, 128),
             lambda d: q.qgemm_f8_wgrad(d(dy), xq, 2, 64, 128), lambda d: q.qmoe_route(d(rows), 2),
             lambda d: q.qmoe_route_backward(rows[:, :8].contiguous(), route, d(route.weight))]
    with fw.dual_level():
        for n, call in enumerate(calls):
            call(lambda t: t)                       # without a tangent
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(ValueError, match="tangent"):
                    call(dual)
                    pytest.fail(f"call {n} was not refused")
    torch.cuda.synchronize()


def test_a_function_with_a_jvp_may_make_the_calls():
    """Rotation alone is linear: its tangent is the rotation of the tangent."""
    q, torch = qg(), torch_cuda()
    fw = torch.autograd.forward_ad
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    f = torch.rand(32, device="cuda")

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return q.qhead_norm_rope(x, None, pos, f)[0]

        @staticmethod
        def jvp(ctx, t):
            return q.qhead_norm_rope(t, None, pos, f)[0]

    x, t = (torch.randn(5, 2, 64, device="cuda") for _ in "xt")
    with fw.dual_level():
        y = fw.unpack_dual(Turn.apply(fw.make_dual(x, t)))
    assert torch.equal(y.primal, q.qhead_norm_rope(x, None, pos, f)[0])
    assert torch.equal(y.tangent, q.qhead_norm_rope(t, None, pos, f)[0])
