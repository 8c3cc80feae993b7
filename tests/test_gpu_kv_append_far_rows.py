"""mla_kv_append on rows whose stride, and whose offsets, pass 32 bits."""
import ctypes

import pytest
import torch

import fp4_kv_cache_sparse_gb300 as mla
from test_gpu_kv_append import DEV, REC, append

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stride,n", [(2 ** 31 + 16, 2), (2 ** 30 + 8, 4)])
@pytest.mark.parametrize("kv_format", list(REC))
def test_rows_far_apart(stride, n, kv_format):
    far = torch.empty((n - 1) * stride + 512, dtype=torch.bfloat16, device=DEV).as_strided((n, 512), (stride, 1))
    x = torch.randn(n, 512, generator=torch.Generator().manual_seed(n)).bfloat16().to(DEV)
    far.copy_(x)
    table = mla.RopeTable(64)
    kw = dict(rope=table, positions=torch.arange(n, dtype=torch.int32, device=DEV) * 1000, offset=448)
    slots = torch.tensor([5, 70, 1, 64][:n], dtype=torch.int32, device=DEV)
    want, err = append(x, slots, 128, kv_format, **kw)
    got, err2 = append(far, slots, 128, kv_format, **kw)
    assert err == err2 == 0 and (got == want).all() and not (got[5] == 0xA5).all()
