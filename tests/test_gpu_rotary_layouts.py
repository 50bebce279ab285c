"""GPU: rotary positions in place on queries and keys whose rows lie between each other's in one buffer give what separate
tensors give, bit for bit; views that share rows are refused."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def fa():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from io_aware_exact_13_gb300 import build

    build.build()
    from io_aware_exact_13_gb300 import fa as mod

    mod.fa_get_device_status()
    return mod


LAYOUTS = {
    # buffer shape, q and k of it
    "packed": ((37, 12, 64), lambda x: (x[:, :8], x[:, 8:10])),
    "heads in turn": ((37, 6, 2, 64), lambda x: (x[:, :, 0], x[:, :, 1])),
    "halves of rows": ((37, 3, 128), lambda x: (x[..., :64], x[..., 64:])),
    "one head": ((37, 9, 64), lambda x: (x[:, 1:], x[:, :1])),
    "batch": ((3, 17, 5, 64), lambda x: (x[:, :, :4].transpose(1, 2), x[:, :, 4:].transpose(1, 2))),
    "heads first": ((3, 6, 17, 64), lambda x: (x[:, :4], x[:, 4:])),
    "tokens in turn": ((3, 4, 34, 64), lambda x: (x[:, :, ::2], x[:, :, 1::2])),
}


@pytest.mark.parametrize("name", LAYOUTS)
def test_in_place_in_one_buffer(fa, name):
    shape, views = LAYOUTS[name]
    torch.manual_seed(len(name))
    x = torch.randn(shape, device=DEV).bfloat16()
    q, k = views(x)
    tokens = (q.shape[0],) if q.dim() == 3 else (q.shape[0], q.shape[2])
    pos = torch.randint(0, 9000, (2, *tokens), dtype=torch.int32, device=DEV)
    inv, axis = fa.rotary_frequencies(32, [20, 12])
    want = fa.rotary(q.clone(), k.clone(), pos, inv, axis)
    rest = x.clone()
    for t, w in zip(views(rest), want):
        t.copy_(w)
    fa.rotary(q, k, pos, inv, axis, inplace=True)
    assert torch.equal(x, rest)  # and what is neither q nor k as it was


def test_views_that_share_rows_are_refused(fa):
    x = torch.randn(37, 12, 64, device=DEV).bfloat16()
    pos = torch.zeros(1, 37, dtype=torch.int32, device=DEV)
    inv, axis = fa.rotary_frequencies(32)
    before = x.clone()
    for q, k in ((x[:, :8], x[:, 7:9]), (x[:, :8], x[:, :8]), (x[:, 3:4], x), (x.view(37, -1)[:, :512].view(37, 8, 64), x.view(37, -1)[:, 480:608].view(37, 2, 64))):
        with pytest.raises(fa.FAError) as e:
            fa.rotary(q, k, pos, inv, axis, inplace=True)
        assert e.value.status == fa.FA_ERR_ARG
        assert torch.equal(x, before)
    assert fa.fa_get_device_status() == fa.FA_OK
