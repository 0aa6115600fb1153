"""CPU: calls of sorting by expert, of products and of dropout that the library or the binding has to refuse before any
device is touched (there is none here)."""
import ctypes
import os

import pytest
import torch

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


class Rows:
    """What the binding looks at of a matrix on the device, without the memory for it."""
    is_cuda = True

    def __init__(self, rows, cols, dtype=torch.bfloat16):
        self.shape, self.dtype = torch.Size((rows, cols)), dtype

    def stride(self):
        return self.shape[1], 1

    def is_contiguous(self):
        return True

    def dim(self):
        return 2

    def numel(self):
        return self.shape[0] * self.shape[1]

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return P

    def get_device(self):
        return 0


HUGE = 1 << 32   # as 32 bits: no rows, which every call accepts


@pytest.fixture
def one_device(monkeypatch):
    monkeypatch.setattr(moe, "_several", False)
    monkeypatch.setattr(moe, "_stream", lambda stream: None)


def test_sizes_past_32_bits_are_refused(lib, one_device):
    tall, wide, idx, f32 = Rows(HUGE, 64), Rows(3, HUGE), Rows(HUGE, 2, torch.int32), torch.float32
    few, one, picks = Rows(3, 64), Rows(3, 1, f32), Rows(3, 1, torch.int32)
    drop = moe.make_dropout(64, torch.bfloat16, 0.5)
    linear = moe.make_linear(Rows(64, 64))
    ffn = moe.make_ffn(*(Rows(64, 64),) * 3)
    norm = moe.make_norm(64, torch.bfloat16)
    rng = Rows(1, 2, torch.int64)
    rng.shape = torch.Size((2,))
    calls = {
        "sort workspace": lambda: moe.moe_sort_workspace(HUGE, 6, 384),
        "sort workspace's experts": lambda: moe.moe_sort_workspace(3, 6, HUGE + 384),
        "sort": lambda: moe.moe_sort(idx, 384, idx, None, flat(385), None),
        "dispatch": lambda: moe.moe_dispatch_forward(tall, Rows(HUGE, 1, torch.int32), few),
        "dispatch to many": lambda: moe.moe_dispatch_forward(few, picks, tall),
        "dispatch of wide rows": lambda: moe.moe_dispatch_forward(wide, picks, wide),
        "dispatch backward": lambda: moe.moe_dispatch_backward(few, Rows(HUGE, 1, torch.int32), tall),
        "combine": lambda: moe.moe_combine_forward(tall, one, picks, few),
        "combine backward": lambda: moe.moe_combine_backward(few, tall, one, picks, tall, one),
        "linear workspace": lambda: moe.moe_linear_workspace(linear, HUGE),
        "linear": lambda: moe.moe_linear_forward(linear, tall, tall, None),
        "linear backward": lambda: moe.moe_linear_backward(linear, tall, tall, None, None, dx=tall),
        "a wide matrix": lambda: moe.make_linear(Rows(64, HUGE + 64)),
        "a tall matrix": lambda: moe.make_linear(Rows(HUGE + 64, 64)),
        "dropout": lambda: moe.moe_dropout_forward(drop, rng, tall, tall),
        "dropout backward": lambda: moe.moe_dropout_backward(drop, rng, tall, tall),
        "dropout of wide rows": lambda: moe.make_dropout(HUGE + 64, torch.bfloat16, 0.5),
        "block workspace": lambda: moe.moe_ffn_workspace(ffn, HUGE),
        "block": lambda: moe.moe_ffn_forward(ffn, tall, tall, None),
        "block backward": lambda: moe.moe_ffn_backward(ffn, tall, tall, None, None, dx=tall),
        "a wide block": lambda: moe.make_ffn(Rows(64, HUGE + 64), Rows(64, HUGE + 64), Rows(HUGE + 64, 64)),
        "norm workspace": lambda: moe.moe_norm_workspace(norm, HUGE),
        "norm": lambda: moe.moe_norm_forward(norm, tall, None, None, tall),
        "norm of wide rows": lambda: moe.make_norm(HUGE + 64, torch.bfloat16),
    }
    for name, call in calls.items():
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == EINVAL, name


def flat(n):
    v = Rows(n, 1, torch.int32)
    v.shape = torch.Size((n,))
    return v
