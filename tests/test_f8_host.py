"""f8 host side: sizes, the host quantizer against the definition, refusals
that need no GPU."""
import numpy as np
import pytest

import f8_util as fu


def _qg():
    import quantized_weight_gemv_amd as q
    q.lib()
    return q


def test_sizes():
    q = _qg()
    assert q.qpacked_bytes_f8(1, 1) == 2048 + 256
    assert q.qpacked_bytes_f8(16, 128) == 2048 + 256
    assert q.qpacked_bytes_f8(17, 129) == 2 * 2 * 2048 + 256
    assert q.qpacked_bytes_f8(4096, 4096) == 4096 * 4096 + 32 * 32
    assert q.qact_bytes_f8(1, 1) == 256 + 256
    assert q.qact_bytes_f8(3, 700) == 3 * 768 + 256       # codes, and 3 x 8 bytes of scales rounded up
    for bad in ((0, 128), (128, 0), (-1, 128), (2 ** 31, 128), (128, 2 ** 20 + 1)):
        assert q.qpacked_bytes_f8(*bad) == 0 and q.qact_bytes_f8(*bad) == 0


@pytest.mark.parametrize("N,K", [(1, 1), (5, 127), (16, 128), (129, 257), (300, 130)])
def test_host_quantizer_follows_the_definition(N, K):
    q = _qg()
    w = fu.weights(N, K, seed=1)
    if N >= 129:
        w[128:, :128] = 0.0                        # a zero block
        w[0, 0] = 448.0 * 2.0 ** -3                # a largest value on the grid's end
        w[1, :8] = np.float32(448.0 * 2.0 ** -3) * (np.arange(8) + 0.5) / 2 ** 17   # subnormal codes and ties
    got, clean = fu.unpack_weights(q.qquantize_f8(w), N, K)
    ref, _ = fu.quantize_weights(w)
    assert clean
    assert np.array_equal(got, ref)


def test_host_quantizer_scale_is_the_smallest_power():
    q = _qg()
    for amax, e in ((448.0, 0), (np.nextafter(np.float32(448), np.float32(500)), 1), (224.0, -1), (1.0, -8),
                    (0.0, 0), (3.4e38, 120), (1e-45, -127), (2.0 ** -118, -126), (2.0 ** -119, -127)):
        w = np.zeros((1, 3), np.float32)
        w[0, 1] = -amax
        packed = q.qquantize_f8(w)
        assert int(packed[2048]) - 127 == e == max(-127, fu.block_exponent(float(np.float32(amax)))), amax


def test_host_quantizer_errors():
    q = _qg()
    w = np.ones((2, 64), np.float32)
    for bad in (np.nan, np.inf, -np.inf):
        w[1, 5] = bad
        with pytest.raises(q.QGError) as e:
            q.qquantize_f8(w)
        assert e.value.status == 4
    with pytest.raises(ValueError):
        q.qquantize_f8(np.ones((2, 64), np.float32), out=np.empty(10, np.uint8))
    with pytest.raises(q.QGError) as e:
        q.qquantize_f8(np.ones((0, 64), np.float32))
    assert e.value.status == 2
    L = q.lib()
    p = np.zeros(4096, np.uint8)
    assert L.qquantize_f8(None, 1, 1, p.ctypes.data, 4096) == 1
    assert L.qquantize_f8(p.ctypes.data, 1, 1, p.ctypes.data, 100) == 5


def test_refusals_before_any_launch():
    """Every check comes before the device is touched, so it runs here too (pointers are never followed)."""
    L = _qg().lib()
    a = 1 << 20   # an aligned address that nothing reads
    assert L.qdequant_f8(None, 1, 1, 0, a, None) == 1
    assert L.qdequant_f8(a, 0, 1, 0, a, None) == 2
    assert L.qdequant_f8(a + 128, 1, 1, 0, a, None) == 3
    assert L.qdequant_f8(a, 1, 1, 0, a + 2, None) == 3
    assert L.qtranspose_f8(a, 1, None or 0, a, None) == 2
    assert L.qtranspose_f8(a, 2 ** 20 + 1, 8, a, None) == 2
    assert L.qtranspose_f8(a, 8, 8, a + 16, None) == 3
    assert L.qact_quantize_f8(a, 3, 8, 1, 8, a, None) == 2
    assert L.qact_quantize_f8(a, 0, 7, 1, 8, a, None) == 2
    assert L.qact_quantize_f8(a + 2, 0, 8, 1, 8, a, None) == 3
    assert L.qact_quantize_f8(a, 0, 8, 0, 8, a, None) == 2
    assert L.qact_dequant_f8(a, 1, 8, -1, a, None) == 2
    for M, K in ((0, 8), (9, 8), (1, 0), (1, 16385)):
        assert L.qgemv_f8(a, a, 1, a, M, 8, K, None) == 2
    assert L.qgemv_f8(a, a + 1, 1, a, 1, 8, 8, None) == 3
    assert L.qgemv_f8(a, None, 1, a, 1, 8, 8, None) == 1
    assert L.qgemm_f8(a, a, a, 5, 1, 8, 8, None) == 2
    assert L.qgemm_f8(a, a + 16, a, 0, 1, 8, 8, None) == 3
    assert L.qgemm_f8(a, a, a + 2, 0, 1, 8, 8, None) == 3
    assert L.qgemm_f8(a, a, a, 0, 2 ** 31, 8, 8, None) == 2
    assert L.qgemm_f8_wgrad(a, a, None, 0, 1, 8, 8, None, None) == 1
    assert L.qgemm_f8_wgrad(a, a, a, 0, 1 << 16, 128, 128, None, None) == 1      # needs a workspace
    assert L.qgemm_f8_wgrad_workspace(1 << 16, 128, 128) > 0
    assert L.qgemm_f8_wgrad(a, a, a, 0, 1 << 16, 128, 128, a + 8, None) == 3
    route = [a, 0, 64, None, 8, 64, 4, 1, a, a, a, a, a, a, None, None]
    for at, value, status in ((0, None, 1), (1, 9, 2), (2, 63, 2), (4, 0, 2), (4, 2 ** 24 + 1, 2), (5, 0, 2),
                              (5, 513, 2), (6, 0, 2), (6, 17, 2), (8, None, 1), (10, a + 2, 3), (12, None, 1),
                              (13, None, 1), (13, a + 1, 3)):
        args = list(route)
        args[at] = value
        if at == 5 and value == 513:
            args[2] = 1024
        assert L.qmoe_route(*args) == status, (at, value)
    assert L.qmoe_route(*route[:4], 100, *route[5:]) == 1                         # needs a workspace
    assert L.qmoe_route(*route[:5], 2, *route[6:]) == 2                           # k above E
    back = [a, 0, 64, None, 8, 64, 4, 1, a, a, a, None, None, a, None]
    for at, value, status in ((13, None, 1), (11, a + 1, 3), (12, a + 2, 3), (6, 65, 2)):
        args = list(back)
        args[at] = value
        assert L.qmoe_route_backward(*args) == status, (at, value)
    moe = [a, 4, a, 8, 2, a, a, a, 0, 64, 64, None]
    for at, value, status in ((0, None, 1), (1, 0, 2), (1, 513, 2), (3, 0, 2), (4, 0, 2), (4, 17, 2), (5, None, 1),
                              (6, a + 2, 3), (8, 4, 2), (9, 0, 2), (10, 2 ** 20 + 1, 2), (7, a + 1, 3)):
        args = list(moe)
        args[at] = value
        assert L.qmoe_gemm_f8(*args) == status, (at, value)
    wg = [a, a, 8, 2, a, a, 4, a, 0, 64, 64, None]
    for at, value, status in ((0, None, 1), (4, None, 1), (6, 513, 2), (7, a + 2, 3), (9, 0, 2)):
        args = list(wg)
        args[at] = value
        assert L.qmoe_gemm_f8_wgrad(*args) == status, (at, value)


def test_binding_refuses_host_tensors_and_bad_sizes():
    torch = pytest.importorskip("torch")
    q = _qg()
    t = torch.zeros(4, 8)
    for call in (lambda: q.qact_quantize_f8(t), lambda: q.qgemv_f8(t, t, 8, 8), lambda: q.qmoe_route(t, 2),
                 lambda: q.qgemm_f8(t, t, 4, 8, 8), lambda: q.qgemm_f8_wgrad(t, t, 4, 8, 8),
                 lambda: q.qmoe_gemm_f8(t, 1, t, 4, t, t, 8, 8), lambda: q.qtranspose_f8(t, 8, 8)):
        with pytest.raises(TypeError):
            call()


def test_limits_of_rows_and_slots():
    """Sizes whose row numbers or gathered offsets would not fit are refused before the device is touched."""
    q = _qg()
    L = q.lib()
    a = 1 << 20
    assert q.qact_bytes_f8(2 ** 30, 1) == 2 ** 30 * 132 and q.qact_bytes_f8(2 ** 30 + 1, 1) == 0
    assert L.qgemm_f8(a, a, a, 0, 2 ** 30 + 1, 8, 8, None) == 2
    assert L.qgemm_f8_wgrad(a, a, a, 0, 2 ** 30 + 1, 8, 8, a, None) == 2
    assert L.qgemm_f8_wgrad_workspace(2 ** 30 + 1, 8, 8) == 0
    assert L.qmoe_gemm_f8(a, 4, a, 2 ** 26 + 1, 16, a, a, a, 0, 8, 8, None) == 2             # slots
    assert L.qmoe_gemm_f8_wgrad(a, a, 2 ** 26 + 1, 16, a, a, 4, a, 0, 8, 8, None) == 2
    assert L.qmoe_gemm_f8(a, 4, a, 2 ** 20, 2, a, a, a, 0, 64, 4096, None) == 2               # 4 GiB of codes
    assert L.qmoe_gemm_f8(a, 4, a, 2 ** 25 - 1, 1, a, a, a, 0, 64, 1, None) == 2
    route = [a, 0, 2 ** 60, None, 8, 64, 4, 1, a, a, a, a, a, a, None, None]
    assert L.qmoe_route(*route) == 2                                                          # rows beyond 63 bits
