"""Norms and rotary positions: gradients past 2^31 elements, tensors without a token, values of the scalings, refusals.  Bounds as
in tests/test_qk.py."""
import pytest
import torch

import block_sparse_flash_ra_gb300 as ra
from tests.test_qk import BF, F4, _c_params, close, forward64, frequencies, turn

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_flash_ra_gb300 import _build
    _build.build()
    yield
    if torch.cuda.is_available():
        torch.cuda.synchronize()
        assert ra.ra_get_device_status() == ra.RA_OK


@gpu
def test_gradients_beyond_32_bits():
    """2^31 elements and more between the first token's rows and the last's, in the inputs and in the gradient: all rows as from
    dense tensors, some against 64 bits, and everything around them left as it was."""
    L, H, D = 1 << 16, 4, 128
    wide = torch.full((1, L, 270, D), 3.0, dtype=BF, device="cuda")
    q = wide[:, :, 100:104]
    q.normal_()
    dy = torch.randn((1, L, H, D), dtype=BF, device="cuda")
    w = (1 + 0.2 * torch.randn(D, generator=torch.Generator().manual_seed(1))).to(BF)
    p = ra.make_qk_params(q, rope=ra.make_rope(128), eps=1e-6, q_weight=w.cuda())
    dense = q.contiguous()
    want, _, dw_want, _ = ra.qk_backward(p, dense, None, dy)
    dx, _, dw, _ = ra.qk_backward(p, q, None, dy, dq=wide[:, :, 200:204])
    assert dx.data_ptr() == wide[:, :, 200:204].data_ptr() and torch.equal(dx, want) and torch.equal(dw, dw_want)
    assert torch.equal(q, dense)
    for lo, hi in ((0, 100), (104, 200), (204, 270)):
        assert (wide[:, :, lo:hi] == 3).all()
    at = torch.tensor([0, 5, 40000, L - 1])
    x64 = dense[:, at].cpu().double().requires_grad_()
    dy64, w64 = dy[:, at].cpu().double(), w.double()
    forward64(x64, at[None], frequencies(D), False, 1.0, w64, 1e-6).backward(dy64)
    r = torch.rsqrt(x64.detach().square().mean(-1, keepdim=True) + 1e-6)
    z, a = (x64.detach() * r).abs(), turn(dy64, at[None], frequencies(D), False, size=True) * w64.abs()
    close(dx[:, at], x64.grad, 2.0 ** -17 * r * (a + z * (a * z).mean(-1, keepdim=True)), "dx")


# ------------------------------------------------------------- no tokens
@pytest.mark.parametrize("shape", [(2, 0, 4, 128), (0, 3, 4, 128), (0, 0, 4, 128), (1, 0, 4, 128), (2, 0, 1, 64)])
def test_strides_of_tensors_without_a_token(shape):
    for x in (torch.empty(shape), torch.empty(shape[:2] + (9, shape[3]))[:, :, 2:2 + shape[2]]):
        assert ra._token_stride(x.shape, x.stride(), "x") >= shape[2] * shape[3]


@gpu
@pytest.mark.parametrize("B,L", [(2, 0), (0, 3), (1, 0)])
def test_calls_without_a_token(B, L):
    x = torch.empty((B, L, 8, 128), dtype=BF, device="cuda")
    q, k, v = x[:, :, :4], x[:, :, 4:6], x[:, :, 6:]
    start = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    p = ra.make_qk_params(q, k, rope=ra.make_rope(64), start=start, eps=1e-6)
    a, b = ra.qk_forward(p, q, k)
    assert a.shape == q.shape and b.shape == k.shape
    for g in (ra.qk_backward(p, q, k, q, k), ra.qk_backward(p, q, k, q, k, dq=q, dk=k)):
        assert g[0].shape == q.shape and g[1].shape == k.shape and (g[2] == 0).all() and (g[3] == 0).all()
    c = ra.new_kv_cache(1, 16, 2, 128, F4)
    assert ra.qk_enter(p, c, q, k, v, table).shape == q.shape
    ra.kv_write(c, k, v, table, start)
    ra.kv_write(c, k.contiguous(), v.contiguous(), table, start)
    assert (c.k_exps == 0).all()


# ------------------------------------------------------------- scalings
def test_values_on_the_ramps():
    """64 rotated values, base 10^4, 8192 positions: pair i turns 8192 / (2 pi) 10^(-i/8) times.  "yarn": the pairs that turn 32
    times and once are 12.88 and 24.92, so the ramp goes from 12 to 25; "bands": 4.12, 3.09, 2.32, 1.74, 1.30 and 0.98 turns for
    pairs 20 to 25."""
    def ratio(**kw):
        r = ra.make_rope(64, 10000.0, device="cpu", trained_length=8192, **kw)
        f = torch.tensor([x % 2 ** 64 / 2 ** 64 for x in r._keep.tolist()], dtype=torch.float64) * 2 * torch.pi
        return (f / frequencies(64)).tolist()
    yarn, bands = ratio(scaling="yarn", factor=16.0), ratio(scaling="bands", factor=8.0)
    for i, x in ((0, 1.0), (12, 1.0), (13, 0.927884615384615), (18, 0.567307692307692), (24, 0.134615384615385), (25, 0.0625), (31, 0.0625)):
        assert abs(yarn[i] - x) < 1e-12
    for i, x in ((20, 1.0), (21, 0.735105597514883), (22, 0.509567132379695), (23, 0.340437143393088), (24, 0.213607544027569), (25, 0.125),
                 (31, 0.125)):
        assert abs(bands[i] - x) < 1e-12


# ------------------------------------------------------------- refusals (no GPU needed)
@pytest.mark.parametrize("apart", [0, 4, 508])
def test_gradients_of_two_weights_in_one_place_are_refused(apart):
    p, M = _c_params(), 1 << 20
    with pytest.raises(ra.RaError, match="dq_weight and dk_weight overlap") as e:
        ra.ra_qk_bwd(p, M, 512, 2 * M, 256, 3 * M, 512, 4 * M, 256, 5 * M, 512, 6 * M, 256, 7 * M, 7 * M + apart, None, stream=0)
    assert e.value.code == ra.RA_ERR_INVALID_ARG
