"""Norms and rotary positions: tensors without a token, refusals."""
import pytest
import torch

import block_sparse_flash_ra_gb300 as ra
from tests.test_qk import BF, F4, _c_params

gpu = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_sparse_flash_ra_gb300 import _build
    _build.build()
    yield
    if torch.cuda.is_available():
        torch.cuda.synchronize()
        assert ra.ra_get_device_status() == ra.RA_OK


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


# ------------------------------------------------------------- refusals (no GPU needed)
@pytest.mark.parametrize("apart", [0, 4, 508])
def test_gradients_of_two_weights_in_one_place_are_refused(apart):
    p, M = _c_params(), 1 << 20
    with pytest.raises(ra.RaError, match="dq_weight and dk_weight overlap") as e:
        ra.ra_qk_bwd(p, M, 512, 2 * M, 256, 3 * M, 512, 4 * M, 256, 5 * M, 512, 6 * M, 256, 7 * M, 7 * M + apart, None, stream=0)
    assert e.value.code == ra.RA_ERR_INVALID_ARG
