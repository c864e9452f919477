"""The wrappers' `stream` argument: what a call on another stream reads stays its own until
the work is done, also when the caller lets go of it at once (GPU)."""
import pytest
import torch

import mixture_experts_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    moe.build()
    assert torch.cuda.is_available()


CALLS = {
    "rope": lambda r, c, x, ids, table, s: moe.rope(r, ids, x, stream=s),
    "append": lambda r, c, x, ids, table, s: c.append(x, x, ids, rotary=r, positions=ids, q=x,
                                                      stream=s),
    "attend": lambda r, c, x, ids, table, s: c.attend(x, table, ids, stream=s),
}


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", list(CALLS))
def test_inputs_let_go_of_are_not_given_away(name, raw):
    B, h, D = 4096, 4, 64
    r = moe.Rotary.build(D, 64)
    c = moe.PagedKVCache.empty(B // 16, 16, h, D, moe.BF16)
    ids = (torch.arange(B, device="cuda") % 16).int()
    table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    CALLS[name](r, c, torch.randn(B, h, D, device="cuda").bfloat16(), ids, table, None)  # warm
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = torch.ones(B, h, D, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)            # the call waits some 50 ms for its turn
    CALLS[name](r, c, x, ids, table, side.cuda_stream if raw else side)
    where = x.data_ptr()
    del x
    others = [torch.empty(B, h, D, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    assert all(o.data_ptr() != where for o in others)
    assert not side.query()                       # the work was indeed still to come
    torch.cuda.synchronize()
    assert moe.coli_device_status() == moe.COLI_OK
