"""Host-side refusals of the drafter layer's calls.  Every call here fails its
checks (or has nothing to do) before CUDA is touched: fake pointers are never
dereferenced on the host."""
import ctypes

import pytest
import torch

from speculative_decoding_pe_gb300 import _native, build

FAKE, MIS = 0x10000, 0x10004
EINVAL, EALIGN = -1, -3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


def _fill(a, **over):
    for name, typ in a._fields_:
        if typ is ctypes.c_void_p:
            setattr(a, name, FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def append_args(**over):
    base = dict(T=14, Hq=64, Hkv=8, D=64, block_size=16, rot_dim=64, interleaved=0, max_pos=100,
                num_blocks=10, q_row=4096, q_head=64, k_row=512, k_head=64, v_row=512, v_head=64)
    return _fill(_native.KvAppendArgs(), **{**base, **over})


def cached_args(**over):
    base = dict(T=14, B=1, Hq=64, Hkv=8, D=64, block_size=16, bt_width=10, scale=0.125,
                num_blocks=10)
    return _fill(_native.AttnCachedArgs(), **{**base, **over})


def prompt_args(**over):
    base = dict(T=14, B=1, Hq=64, Hkv=8, D=64, scale=0.125, q_row=4096, q_head=64, k_row=512,
                k_head=64, v_row=512, v_head=64)
    return _fill(_native.AttnPromptArgs(), **{**base, **over})


@pytest.mark.parametrize("over, rc", [
    (dict(T=-1), EINVAL), (dict(Hq=63), EINVAL), (dict(Hkv=0), EINVAL), (dict(D=96), EINVAL),
    (dict(T=1 << 27), EINVAL), (dict(block_size=8), EINVAL), (dict(block_size=24), EINVAL), (dict(num_blocks=0), EINVAL),
    (dict(num_blocks=1 << 60), EINVAL), (dict(rot_dim=0), EINVAL), (dict(rot_dim=48), EINVAL),
    (dict(rot_dim=96), EINVAL), (dict(max_pos=0), EINVAL), (dict(q=None), EINVAL),
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(positions=None), EINVAL),
    (dict(slots=None), EINVAL), (dict(rope=None), EINVAL), (dict(cache=None), EINVAL),
    (dict(q_out=None), EINVAL), (dict(err=None), EINVAL), (dict(q=MIS), EALIGN),
    (dict(k_out=MIS), EALIGN), (dict(cache=MIS), EALIGN), (dict(rope=MIS), EALIGN),
    (dict(q_row=4100), EALIGN), (dict(k_head=68), EALIGN), (dict(v_row=-8), EALIGN),
    (dict(T=0, q=None), 0)])
def test_append_refusals(lib, over, rc):
    assert lib.pe_kv_append(ctypes.byref(append_args(**over)), None) == rc


@pytest.mark.parametrize("over, rc", [
    (dict(n=-1), EINVAL), (dict(n=1 << 26), EINVAL), (dict(D=32), EINVAL), (dict(bs=20), EINVAL), (dict(Hkv=0), EINVAL),
    (dict(nb=0), EINVAL), (dict(cache=None), EINVAL), (dict(slots=None), EINVAL),
    (dict(err=None), EINVAL), (dict(cache=MIS), EALIGN), (dict(k=MIS), EALIGN),
    (dict(v=MIS), EALIGN), (dict(n=0, cache=None), 0)])
def test_read_refusals(lib, over, rc):
    a = {**dict(cache=FAKE, nb=10, bs=16, Hkv=8, D=64, slots=FAKE, n=4, k=FAKE, v=FAKE, err=FAKE), **over}
    assert lib.pe_kv_read(*a.values(), None) == rc


COMMON = [
    (dict(T=-1), EINVAL), (dict(B=0), EINVAL), (dict(B=2049), EINVAL), (dict(Hq=65), EINVAL),
    (dict(Hq=129, Hkv=1), EINVAL), (dict(D=80), EINVAL), (dict(scale=float("nan")), EINVAL),
    (dict(scale=float("inf")), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-0.125), EINVAL),
    (dict(T=15, B=2, offsets=None), EINVAL),
    (dict(q=None), EINVAL), (dict(out=None), EINVAL), (dict(workspace=None), EINVAL),
    (dict(err=None), EINVAL), (dict(q=MIS), EALIGN), (dict(out=MIS), EALIGN),
    (dict(workspace=MIS), EALIGN), (dict(T=0, q=None), 0)]


@pytest.mark.parametrize("over, rc", COMMON + [
    (dict(block_size=0), EINVAL), (dict(block_size=30), EINVAL), (dict(bt_width=0), EINVAL),
    (dict(bt_width=1 << 28), EINVAL), (dict(num_blocks=0), EINVAL), (dict(cache=None), EINVAL),
    (dict(block_table=None), EINVAL), (dict(positions=None), EINVAL), (dict(cache=MIS), EALIGN)])
def test_cached_refusals(lib, over, rc):
    assert lib.pe_attn_cached(ctypes.byref(cached_args(**over)), None) == rc


@pytest.mark.parametrize("over, rc", COMMON + [
    (dict(k=None), EINVAL), (dict(v=None), EINVAL), (dict(k=MIS), EALIGN), (dict(v=MIS), EALIGN),
    (dict(q_row=-8), EINVAL), (dict(k_row=1 << 31), EINVAL), (dict(v_head=60), EALIGN)])
def test_prompt_refusals(lib, over, rc):
    assert lib.pe_attn_prompt(ctypes.byref(prompt_args(**over)), None) == rc


def test_null_arguments(lib):
    for f in (lib.pe_kv_append, lib.pe_attn_cached, lib.pe_attn_prompt):
        assert f(None, None) == EINVAL


def test_workspace_bytes(lib):
    assert lib.pe_workspace_bytes_attn(64) > 0
    assert lib.pe_workspace_bytes_attn(128) > lib.pe_workspace_bytes_attn(64)
    assert lib.pe_workspace_bytes_attn(96) == 0


def test_binding_refuses_host_tensors(lib):
    cpu = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 8, 1, 18 * 64, dtype=torch.uint8)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        _native.kv_append(cpu, cpu, cpu, i, i.long(), torch.zeros(9, 64), cache, cpu, i)
    with pytest.raises(ValueError):
        _native.kv_read(cache, i.long(), cpu, cpu, i)
    with pytest.raises(ValueError):
        _native.attn_cached(cpu, cache, i.view(2, 2), None, i, None, cpu, i, i)
    with pytest.raises(ValueError):
        _native.attn_prompt(cpu, cpu, cpu, i, cpu, i, i)
    with pytest.raises(ValueError):
        _native.new_kv_cache(4, 17, 8, 64, device="cpu")


def test_cache_and_rope_tables():
    assert _native.new_kv_cache(3, 32, 2, 64, device="cpu").shape == (3, 2, 2, 1152)
    r = _native.rope_table(70000, 64, device="cpu")
    p = torch.arange(70000, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32).double() / 32)
    assert r.shape == (70000, 64) and r.dtype == torch.float32
    # each entry is its 64-bit value rounded once (half a step, 2^-24 of at most 1)
    assert float((r[:, :32].double() - p.cos()).abs().max()) <= 2.0 ** -24
    assert float((r[:, 32:].double() - p.sin()).abs().max()) <= 2.0 ** -24
