"""CPU: calls of sorting by expert, of products and of dropout that the library or the binding has to refuse before any
device is touched (there is none here)."""
import ctypes
import os

import pytest

import mixture_experts_ffn_gemv_amd as moe

P = 1 << 20   # an aligned stand-in for a device pointer: never followed
EINVAL, ESCRATCH = moe.MOE_EINVAL, moe.MOE_ESCRATCH


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(moe.LIB_PATH):
        pytest.skip("libmoe.so not built")
    return moe.lib()


@pytest.mark.parametrize("m", [3, 1000, 9000])   # by one launch and by two
def test_sort_onto_its_picks_is_refused(lib, m):
    # every workgroup reads picks that others' results would have taken the place of
    topk, experts = 6, 384
    n, far = 4 * m * topk, 1 << 24
    size = ctypes.c_size_t()
    assert lib.moe_sort_workspace(m, topk, experts, ctypes.byref(size)) == moe.MOE_OK

    def call(row_of=P + far, pick_of=P + 2 * far, offsets=P + 3 * far, work_bytes=size.value):
        return lib.moe_sort(P, m, topk, experts, row_of, pick_of, offsets, P + 4 * far, work_bytes, None)

    for at in (P, P + 4, P + n - 4, P - n + 4):
        assert call(row_of=at) == EINVAL and call(pick_of=at) == EINVAL, at - P
    for at in (P, P + n - 4, P - 4 * experts):
        assert call(offsets=at) == EINVAL, at - P
    if size.value:
        assert call(row_of=P, work_bytes=size.value - 1) == ESCRATCH
