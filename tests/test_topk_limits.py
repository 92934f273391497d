"""Which sizes the scores' alternatives are refused at: the header says above 16 million 16-bit or 8 million 32-bit columns, for
any number of them.  No rows, so that the checks are all that runs."""
import ctypes as C

import pytest

from sinkhorn_point_cloud_gb300 import binding, build

P = C.c_void_p(64)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def asked(lib, V, K, dtype):
    return lib.sot_token_topk(P, 0, V, V, dtype, 1.0, P, binding.SOT_I64, K, P, P, P, P, P, None)


@pytest.mark.parametrize("K", [1, 64, 256, 257, 512, 513, 1000, 1024])
@pytest.mark.parametrize("dtype,limit", [(binding.SOT_BF16, 16_000_000), (binding.SOT_F16, 16_000_000), (binding.SOT_F32, 8_000_000)])
def test_alternatives_fit_up_to_the_stated_columns(lib, K, dtype, limit):
    for V in (1, 7, 1000, 5000, 131072, 600001, limit // 4 + 1, limit // 2 + 1, limit - limit // 8, limit - 3, limit):
        assert asked(lib, V, K, dtype) == binding.SOT_OK, V
    for V in (2 * limit, 4 * limit + 1):
        assert asked(lib, V, K, dtype) == binding.SOT_ERR_UNSUPPORTED, V
        assert b"do not fit" in lib.sot_last_error()
    assert asked(lib, 4 * limit, 0, dtype) == binding.SOT_OK  # without alternatives
