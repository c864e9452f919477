"""Refusals of the attention-side entry points and wrappers (CPU only)."""
import math

import pytest

import mixture_experts_gb300 as moe
from mixture_experts_gb300 import _build

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return moe.lib()


# ---- rotary table -----------------------------------------------------------------------
@pytest.mark.parametrize("field,value", [
    ("scaling", 16), ("scaling", 18), ("scaling", 20), ("base", 1.0), ("base", 0.5),
    ("beta_slow", 0.0), ("beta_slow", -1.0), ("beta_fast", 1.0), ("original_positions", 0),
    ("factor", 0.0), ("beta_slow", math.nan)])
def test_yarn_over_the_index_rejects(field, value):
    cfg = moe.coli_rope_config(64, moe.ROPE_YARN_INDEX, 4096, 10000.0, 4.0, 32.0, 1.0, 1.0)
    setattr(cfg, field, value)
    assert moe.coli_rope_table(cfg, 128, FAKE, stream=0) == moe.COLI_EINVAL
    assert moe.last_error()


# ---- devices ----------------------------------------------------------------------------
class Standin:
    """What the wrappers ask of a tensor, on any device index; nothing is behind it."""
    is_cuda = True

    def __init__(self, shape, dtype, dev):
        self.shape, self.dtype, self._dev, self.device = shape, dtype, dev, f"cuda:{dev}"

    def get_device(self):
        return self._dev

    def dim(self):
        return len(self.shape)

    def stride(self):
        s = [1]
        for n in self.shape[:0:-1]:
            s.append(s[-1] * n)
        return tuple(s[::-1])

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


@pytest.fixture
def devices(monkeypatch):
    """Makers of stand-ins, device 0 current, and a library that must not be called."""
    import torch
    moe._t()

    def called():
        raise AssertionError("the library was called")
    monkeypatch.setattr(moe, "lib", called)
    monkeypatch.setattr(moe, "_current_device", lambda: 0, raising=False)

    def rows(dev, heads=2):
        return Standin((3, heads, 64), torch.bfloat16, dev)

    def ids(dev):
        return Standin((3,), torch.int32, dev)

    def cache(dev, scale_dev=None):
        k, v = (Standin((4, 2, 16, 64), torch.uint8, dev) for _ in range(2))
        s = [Standin((4, 2, 16, 4), torch.uint8, dev if scale_dev is None else scale_dev)
             for _ in range(2)]
        return moe.PagedKVCache(k, v, *s, head_dim=64)

    def rotary(dev):
        return moe.Rotary(Standin((8, 32, 2), torch.float32, dev))

    def table(dev):
        return Standin((3, 4), torch.int32, dev)
    return rows, ids, cache, rotary, table


def test_wrappers_refuse_other_devices(devices):
    rows, ids, cache, rotary, table = devices
    c, r = cache(0), rotary(0)
    other = cache(1)
    for bad in (
            lambda: moe.rope(rotary(1), ids(1), rows(1)), lambda: moe.rope(r, ids(0), rows(1)),
            lambda: moe.rope(rotary(1), ids(0), rows(0)),
            lambda: moe.rope(r, ids(1), rows(0), q_out=rows(0)),
            lambda: moe.rope(r, ids(0), rows(0), rows(1), q_out=rows(0)),
            lambda: moe.rope(r, ids(0), rows(0), q_out=rows(1)),
            lambda: moe.rope(r, ids(0), rows(0), rows(0), q_out=rows(0), k_out=rows(1)),
            lambda: cache(0, 1), lambda: other.append(rows(1), rows(1), ids(1)),
            lambda: c.append(rows(1), rows(0), ids(0)), lambda: c.append(rows(0), rows(1), ids(0)),
            lambda: c.append(rows(0), rows(0), ids(1)),
            lambda: c.append(rows(0), rows(0), ids(0), rotary=rotary(1), positions=ids(0)),
            lambda: c.append(rows(0), rows(0), ids(0), rotary=r, positions=ids(1)),
            lambda: c.append(rows(0), rows(0), ids(0), rotary=r, positions=ids(0), q=rows(1)),
            lambda: c.append(rows(0), rows(0), ids(0), rotary=r, positions=ids(0), q=rows(0),
                             q_out=rows(1)),
            lambda: other.read(ids(1)), lambda: c.read(ids(1)),
            lambda: other.attend(rows(1), table(1), ids(1)),
            lambda: c.attend(rows(1), table(0), ids(0)),
            lambda: c.attend(rows(0), table(1), ids(0), out=rows(0)),
            lambda: c.attend(rows(0), table(0), ids(0), out=rows(1)),
            lambda: c.attend(rows(0), table(0), ids(1), out=rows(0))):
        with pytest.raises(ValueError, match="cuda:|device"):
            bad()


def test_pools_of_two_devices_are_refused(devices):
    import torch
    k, v = (Standin((4, 2, 16, 64), torch.bfloat16, d) for d in (0, 1))
    with pytest.raises(ValueError, match="one device"):
        moe.PagedKVCache(k, v)


# ---- alignment ---------------------------------------------------------------------------
@pytest.mark.parametrize("off", [1, 2, 3])
def test_ids_and_results_have_to_be_aligned(off):
    """A 32-bit vector off its boundary would fault in the kernel."""
    odd = FAKE + off
    c = moe.coli_kv_cache(FAKE, FAKE, FAKE, FAKE, 8, 16, 2, 64, moe.BF16)
    r = moe.coli_rotary(FAKE, 100, 64, moe.ROPE_HALF, 0)
    cfg = moe.coli_attn_config(4, 0, 0.125)

    def attend(table=FAKE, lens=FAKE, lse=FAKE):
        return moe.coli_paged_attention(c, cfg, FAKE, 256, 2, table, 4, lens, 2 * FAKE, 256, lse,
                                        FAKE, 1 << 40, stream=0)
    for what, call in (
            ("positions", lambda: moe.coli_rope_apply(r, odd, 4, 64, moe.BF16, FAKE, 128, 2, FAKE,
                                                      128, stream=0)),
            ("positions", lambda: moe.coli_kv_append(c, FAKE, 128, FAKE, 128, FAKE, 4, r, odd,
                                                     stream=0)),
            ("slots", lambda: moe.coli_kv_append(c, FAKE, 128, FAKE, 128, odd, 4, stream=0)),
            ("slots", lambda: moe.coli_kv_read(c, odd, 4, FAKE, 128, FAKE, 128, stream=0)),
            ("block_table", lambda: attend(table=odd)), ("seq_lens", lambda: attend(lens=odd)),
            ("lse", lambda: attend(lse=odd))):
        assert call() == moe.COLI_EINVAL, what
        assert what in moe.last_error()


# ---- ranks and names ---------------------------------------------------------------------
def test_wrappers_refuse_other_ranks_with_a_value_error(devices):
    import torch
    rows, ids, cache, rotary, table = devices
    c, r = cache(0), rotary(0)

    def flat(*shape, dtype=torch.bfloat16):
        return Standin(shape, dtype, 0)
    for bad in (
            lambda: moe.rope(r, ids(0), flat(64)),
            lambda: moe.rope(r, ids(0), rows(0), flat(64), q_out=rows(0)),
            lambda: moe.rope(r, ids(0), rows(0), flat(), q_out=rows(0)),
            lambda: c.append(flat(), rows(0), ids(0)), lambda: c.append(flat(3), rows(0), ids(0)),
            lambda: c.append(rows(0), flat(3), ids(0)),
            lambda: c.append(rows(0), rows(0), ids(0), rotary=r, positions=ids(0), q=flat(3)),
            lambda: c.read(flat(dtype=torch.int32)), lambda: c.read(flat(3, 1, dtype=torch.int32)),
            lambda: c.attend(flat(3), table(0), ids(0)), lambda: c.attend(flat(), table(0), ids(0)),
            lambda: moe.Rotary(Standin((8, 32, 2), torch.float32, 0), "halves"),
            lambda: moe.Rotary(Standin((8, 32, 2), torch.float32, 0), 2)):
        with pytest.raises(ValueError):
            bad()
