"""The attention-side entry points reject bad arguments before anything is
launched, and the 64-bit forms the GPU tests compare with agree with torch's
own types (CPU only)."""
import ctypes
import math
import os
import sys

import pytest
import torch

import mixture_experts_gb300 as moe
from mixture_experts_gb300 import _build, inputs

sys.path.insert(0, os.path.dirname(__file__))
import attn_ref  # noqa: E402

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return moe.lib()


def cache(**kw):
    c = moe.coli_kv_cache(FAKE, FAKE, FAKE, FAKE, 8, 16, 2, 64, moe.BF16)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def rotary(**kw):
    r = moe.coli_rotary(FAKE, 100, 64, moe.ROPE_HALF, 0)
    for n, v in kw.items():
        setattr(r, n, v)
    return r


BAD_CACHES = [dict(dtype=moe.I4G128), dict(dtype=9), dict(head_dim=60), dict(head_dim=0),
              dict(head_dim=264), dict(dtype=moe.MXFP8, head_dim=80), dict(page_size=8),
              dict(page_size=24), dict(page_size=8192), dict(n_kv_heads=0), dict(n_kv_heads=257),
              dict(n_pages=0), dict(n_pages=1 << 27), dict(k=None), dict(v=FAKE + 8),
              dict(dtype=moe.MXFP4, k_scale=None), dict(dtype=moe.MXFP8, v_scale=FAKE + 2)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_bad_caches_are_rejected_by_every_call(bad):
    c = cache(**bad)
    assert moe.coli_kv_append(c, FAKE, 128, FAKE, 128, FAKE, 4, stream=0) == moe.COLI_EINVAL
    assert moe.last_error()
    assert moe.coli_kv_read(c, FAKE, 4, FAKE, 128, FAKE, 128, stream=0) == moe.COLI_EINVAL
    cfg = moe.coli_attn_config(4, 0, 0.125)
    assert moe.coli_paged_attention(c, cfg, FAKE, 256, 2, FAKE, 4, FAKE, FAKE, 256, None, FAKE,
                                    1 << 30, stream=0) == moe.COLI_EINVAL
    assert moe.coli_paged_attention_scratch_bytes(c, 2, 4) == 0


def test_null_structs():
    assert moe.coli_rope_table(None, 4, FAKE, stream=0) == moe.COLI_EINVAL
    assert moe.coli_rope_apply(None, FAKE, 4, 64, moe.BF16, FAKE, 128, 2, FAKE, 128,
                               stream=0) == moe.COLI_EINVAL
    assert moe.coli_kv_append(None, FAKE, 128, FAKE, 128, FAKE, 4, stream=0) == moe.COLI_EINVAL
    assert moe.coli_kv_read(None, FAKE, 4, FAKE, 128, None, 0, stream=0) == moe.COLI_EINVAL
    assert moe.coli_paged_attention(cache(), None, FAKE, 256, 2, FAKE, 4, FAKE, FAKE, 256,
                                    stream=0) == moe.COLI_EINVAL


@pytest.mark.parametrize("field,value", [
    ("rot_dim", 0), ("rot_dim", 7), ("rot_dim", 258), ("scaling", 4), ("scaling", -1),
    ("base", 0.0), ("base", math.inf), ("amplitude", math.nan), ("factor", 0.0),
    ("factor", -2.0), ("original_positions", 0), ("beta_fast", 1.0)])
def test_rope_table_rejects(field, value):
    cfg = moe.coli_rope_config(64, moe.ROPE_YARN, 4096, 10000.0, 4.0, 32.0, 1.0, 1.0)
    setattr(cfg, field, value)
    assert moe.coli_rope_table(cfg, 128, FAKE, stream=0) == moe.COLI_EINVAL
    assert moe.last_error()


def test_rope_table_rejects_sizes():
    cfg = moe.coli_rope_config(64, 0, 0, 10000.0, 0.0, 0.0, 0.0, 1.0)
    for n, t in ((0, FAKE), (1 << 26, FAKE), (16, None), (16, FAKE + 4)):
        assert moe.coli_rope_table(cfg, n, t, stream=0) == moe.COLI_EINVAL
    cfg = moe.coli_rope_config(2, moe.ROPE_NTK, 0, 10000.0, 4.0, 0.0, 0.0, 1.0)
    assert moe.coli_rope_table(cfg, 16, FAKE, stream=0) == moe.COLI_EINVAL


@pytest.mark.parametrize("kw,word", [
    (dict(rotary=rotary(table=None)), "table"), (dict(rotary=rotary(table=FAKE + 8)), "table"),
    (dict(rotary=rotary(rot_dim=66)), "rot_dim"), (dict(rotary=rotary(rot_dim=3)), "rot_dim"),
    (dict(rotary=rotary(layout=2)), "layout"), (dict(rotary=rotary(inverse=2)), "inverse"),
    (dict(rotary=rotary(n_positions=0)), "n_positions"), (dict(positions=None), "positions"),
    (dict(T=-1), "T="), (dict(T=(1 << 24) + 1), "T="), (dict(head_dim=100), "head_dim"),
    (dict(act=moe.MXFP8), "act"), (dict(q=None), "q"), (dict(q=FAKE + 4), "aligned"),
    (dict(q_stride=132), "aligned"), (dict(q_stride=64), "stride"), (dict(n_q_heads=0), "heads"),
    (dict(n_q_heads=1025), "heads"), (dict(q_out=None), "q_out"),
    (dict(q_out_stride=8), "stride"), (dict(k_out=None), "k_out"), (dict(n_kv_heads=0), "heads"),
    (dict(q_out=FAKE, q_stride=256), "place")])
def test_rope_apply_rejects(kw, word):
    a = dict(rotary=rotary(), positions=FAKE, T=4, head_dim=64, act=moe.BF16, q=FAKE,
             q_stride=128, n_q_heads=2, q_out=2 * FAKE, q_out_stride=128, k=3 * FAKE,
             k_stride=64, n_kv_heads=1, k_out=4 * FAKE, k_out_stride=64)
    a.update(kw)
    assert moe.coli_rope_apply(**a, stream=0) == moe.COLI_EINVAL
    assert word in moe.last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(slots=None), "slots"), (dict(T=-1), "T="), (dict(k=None), "k must"),
    (dict(v=FAKE + 2), "aligned"), (dict(k_stride=100), "aligned"), (dict(v_stride=64), "stride"),
    (dict(rotary=None), "rotary"), (dict(positions=None), "positions"),
    (dict(rotary=rotary(rot_dim=128)), "rot_dim"), (dict(n_q_heads=0), "heads"),
    (dict(q_out=None), "q_out"), (dict(q_stride=100), "aligned"),
    (dict(q_out=FAKE, q_out_stride=512), "place")])
def test_append_rejects(kw, word):
    a = dict(cache=cache(), k=FAKE, k_stride=128, v=FAKE, v_stride=128, slots=FAKE, T=4,
             rotary=rotary(), positions=FAKE, q=FAKE, q_stride=256, n_q_heads=4, q_out=2 * FAKE,
             q_out_stride=256)
    a.update(kw)
    assert moe.coli_kv_append(**a, stream=0) == moe.COLI_EINVAL
    assert word in moe.last_error()


def test_read_rejects():
    for a in ((None, 4, FAKE, 128, FAKE, 128), (FAKE, -1, FAKE, 128, FAKE, 128),
              (FAKE, 4, None, 0, None, 0), (FAKE, 4, FAKE + 8, 128, None, 0),
              (FAKE, 4, FAKE, 120, None, 0), (FAKE, 4, None, 0, FAKE, 100)):
        assert moe.coli_kv_read(cache(), *a, stream=0) == moe.COLI_EINVAL


@pytest.mark.parametrize("kw,word", [
    (dict(B=-1), "B="), (dict(B=65536), "B="), (dict(q=None), "q must"),
    (dict(q_stride=128), "stride"), (dict(out=FAKE), "must not be q"),
    (dict(out=FAKE + 4), "aligned"),
    (dict(block_table=None), "block_table"), (dict(seq_lens=None), "seq_lens"),
    (dict(max_pages=0), "max_pages"), (dict(max_pages=1 << 27), "max_pages"),
    (dict(cfg=moe.coli_attn_config(3, 0, 1.0)), "multiple"),
    (dict(cfg=moe.coli_attn_config(0, 0, 1.0)), "heads"),
    (dict(cfg=moe.coli_attn_config(4, -1, 1.0)), "window"),
    (dict(cfg=moe.coli_attn_config(4, 0, math.inf)), "scale"),
    (dict(cfg=moe.coli_attn_config(4, 0, math.nan)), "scale")])
def test_attention_rejects(kw, word):
    a = dict(cache=cache(), cfg=moe.coli_attn_config(4, 0, 0.125), q=FAKE, q_stride=256, B=2,
             block_table=FAKE, max_pages=4, seq_lens=FAKE, out=2 * FAKE, out_stride=256,
             scratch=FAKE, scratch_bytes=1 << 40)
    a.update(kw)
    assert moe.coli_paged_attention(**a, stream=0) == moe.COLI_EINVAL
    assert word in moe.last_error()


def test_empty_batches_are_fine_without_a_gpu():
    assert moe.coli_rope_apply(rotary(), FAKE, 0, 64, moe.BF16, FAKE, 128, 2, FAKE, 128,
                               stream=0) == moe.COLI_OK
    assert moe.coli_kv_append(cache(), FAKE, 128, FAKE, 128, FAKE, 0, stream=0) == moe.COLI_OK
    assert moe.coli_kv_read(cache(), FAKE, 0, FAKE, 128, None, 0, stream=0) == moe.COLI_OK
    assert moe.coli_paged_attention(cache(), moe.coli_attn_config(4, 0, 1.0), FAKE, 256, 0, FAKE,
                                    1, FAKE, FAKE, 256, stream=0) == moe.COLI_OK


def test_struct_sizes_match_the_header(tmp_path):
    import shutil
    import subprocess
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ("coli_rope_config", "coli_rotary", "coli_kv_cache", "coli_attn_config")
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "coli_moe.h"\nint main(void){'
                   + "".join(f'printf("%zu ", sizeof({n}));' for n in names) + "return 0;}")
    subprocess.run([cc, "-I", os.path.dirname(moe.HEADER), str(src), "-o", str(tmp_path / "s")],
                   check=True)
    got = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True).stdout.split()
    assert [int(x) for x in got] == [ctypes.sizeof(getattr(moe, n)) for n in names]


def test_python_wrappers_reject_cpu_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.Rotary(torch.zeros(8, 32, 2))
    with pytest.raises(ValueError):
        moe.PagedKVCache(torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64))
    with pytest.raises(ValueError):
        moe._head_rows("x", x, 2, 64, torch.bfloat16)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_reference_quantiser_agrees_with_the_framework_inputs(fmt):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 96, generator=g) * torch.exp2(torch.randint(-30, 30, (40, 1),
                                                                    generator=g).float())
    x[3] = 0
    codes, scales = attn_ref.quantise(x, fmt)
    want_c, want_s = inputs.quantize_mx(x, fmt)
    assert torch.equal(codes, want_c) and torch.equal(scales, want_s)
    if fmt == "mxfp8":
        want = codes.view(torch.float8_e4m3fn).double().unflatten(-1, (-1, 32))
        want = (want * torch.exp2(scales.double() - 127)[..., None]).flatten(-2)
        assert torch.equal(attn_ref.decode(codes, scales, fmt), want)


def test_reference_e4m3_values_are_torch_s():
    codes = torch.arange(256, dtype=torch.uint8).reshape(8, 32)
    got = attn_ref.decode(codes, torch.full((8, 1), 127, dtype=torch.uint8), "mxfp8")
    want = codes.view(torch.float8_e4m3fn).double()
    assert torch.equal(got.nan_to_num(1e9), want.nan_to_num(1e9))
