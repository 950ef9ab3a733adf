"""Host-side refusals of the filtered sampling's and the bounded cache's calls.
Every call here fails its checks (or has nothing to do) before CUDA is touched:
fake pointers are never dereferenced on the host."""
import ctypes

import pytest
import torch

from speculative_decoding_pe_gb300 import _native, build

FAKE, MIS = 0x10000, 0x10004
EINVAL, EDTYPE, EALIGN = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _native.load()


def fill(a, **over):
    for name, typ in a._fields_:
        if typ is ctypes.c_void_p:
            setattr(a, name, FAKE)
    for k, v in over.items():
        setattr(a, k, v)
    return ctypes.byref(a)


SAMPLE = dict(n=6, requests=2, rows=6, V=1000, dtype=1, row_stride=1000)
VERIFY = dict(B=2, Kp=3, V=1000, dtype=1, target_stride=1000, draft_stride=1000)
WEIGH = dict(T=14, B=1, Hq=64, Hkv=8, D=64, block_size=16, bt_width=10, scale=0.125, num_blocks=10)
EVICT = dict(B=2, Hkv=8, D=64, block_size=16, bt_width=10, dst_width=4, max_keep=50, sinks=0, recent=0, num_blocks=30)


@pytest.mark.parametrize("over, rc", [
    (dict(n=-1), EINVAL), (dict(n=7), EINVAL), (dict(requests=0), EINVAL), (dict(requests=4), EINVAL), (dict(V=0), EINVAL),
    (dict(V=262145, row_stride=262152), EINVAL), (dict(rows=-1), EINVAL), (dict(rows=0), EINVAL), (dict(rows=5, sample_idx=None), EINVAL),
    (dict(n=(1 << 27) + 1), EINVAL), (dict(dtype=2), EDTYPE), (dict(row_stride=992), EINVAL), (dict(row_stride=1004), EALIGN),
    (dict(row_stride=1 << 62), EINVAL), (dict(logits=None), EINVAL), (dict(u=None), EINVAL), (dict(out_tokens=None), EINVAL),
    (dict(err=None), EINVAL), (dict(logits=MIS), EALIGN), (dict(n=0, logits=None), 0)])
def test_sample_refusals(lib, over, rc):
    assert lib.pe_draft_sample(fill(_native.DraftSampleArgs(), **{**SAMPLE, **over}), None) == rc


@pytest.mark.parametrize("over, rc", [
    (dict(B=-1), EINVAL), (dict(Kp=-1), EINVAL), (dict(Kp=256), EINVAL), (dict(V=0), EINVAL), (dict(V=1 << 19), EINVAL),
    (dict(B=1 << 26), EINVAL), (dict(dtype=-1), EDTYPE), (dict(target_stride=999), EINVAL), (dict(draft_stride=999), EINVAL),
    (dict(target_stride=1001), EALIGN), (dict(draft_stride=1001), EALIGN), (dict(target_logits=None), EINVAL),
    (dict(draft_logits=None), EINVAL), (dict(in_tokens=None), EINVAL), (dict(u_accept=None), EINVAL), (dict(u_draw=None), EINVAL),
    (dict(accepted_len=None), EINVAL), (dict(bonus_token=None), EINVAL), (dict(workspace=None), EINVAL), (dict(err=None), EINVAL),
    (dict(target_logits=MIS), EALIGN), (dict(draft_logits=MIS), EALIGN), (dict(workspace=MIS), EALIGN),
    (dict(B=0, target_logits=None), 0)])
def test_verify_refusals(lib, over, rc):
    assert lib.pe_verify_filtered(fill(_native.VerifyFilteredArgs(), **{**VERIFY, **over}), None) == rc


@pytest.mark.parametrize("over, rc", [
    (dict(T=-1), EINVAL), (dict(B=0), EINVAL), (dict(B=2049), EINVAL), (dict(Hq=63), EINVAL), (dict(Hq=129, Hkv=1), EINVAL),
    (dict(D=96), EINVAL), (dict(block_size=24), EINVAL), (dict(bt_width=0), EINVAL), (dict(bt_width=1 << 28), EINVAL),
    (dict(num_blocks=0), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
    (dict(T=15, B=2, offsets=None), EINVAL), (dict(T=1 << 27), EINVAL), (dict(B=2048, Hq=64, Hkv=64), EINVAL),
    (dict(q=None), EINVAL), (dict(cache=None), EINVAL), (dict(block_table=None), EINVAL), (dict(positions=None), EINVAL),
    (dict(out=None), EINVAL), (dict(workspace=None), EINVAL), (dict(err=None), EINVAL), (dict(q=MIS), EALIGN),
    (dict(cache=MIS), EALIGN), (dict(mass=MIS), EALIGN), (dict(out=MIS), EALIGN), (dict(workspace=MIS), EALIGN),
    (dict(T=0, q=None), 0)])
def test_weigh_refusals(lib, over, rc):
    assert lib.pe_kv_weigh(fill(_native.KvWeighArgs(), **{**WEIGH, **over}), None) == rc


@pytest.mark.parametrize("over, rc", [
    (dict(B=-1), EINVAL), (dict(Hkv=0), EINVAL), (dict(D=80), EINVAL), (dict(block_size=0), EINVAL), (dict(bt_width=0), EINVAL),
    (dict(dst_width=0), EINVAL), (dict(max_keep=0), EINVAL), (dict(sinks=-1), EINVAL), (dict(recent=-1), EINVAL),
    (dict(num_blocks=0), EINVAL), (dict(num_blocks=1 << 60), EINVAL), (dict(bt_width=1 << 28), EINVAL), (dict(dst_width=1 << 28), EINVAL),
    (dict(B=1 << 22), EINVAL), (dict(cache=None), EINVAL), (dict(mass=None), EINVAL), (dict(block_table=None), EINVAL),
    (dict(dst_table=None), EINVAL), (dict(lengths=None), EINVAL), (dict(keep=None), EINVAL), (dict(kept=None), EINVAL),
    (dict(out_lengths=None), EINVAL), (dict(err=None), EINVAL), (dict(cache=MIS), EALIGN), (dict(mass=MIS), EALIGN),
    (dict(B=0, cache=None), 0)])
def test_evict_refusals(lib, over, rc):
    assert lib.pe_kv_evict(fill(_native.KvEvictArgs(), **{**EVICT, **over}), None) == rc


def test_null_arguments(lib):
    for name in ("pe_draft_sample", "pe_verify_filtered", "pe_kv_weigh", "pe_kv_evict"):
        assert getattr(lib, name)(None, None) == EINVAL


def test_workspace_bytes(lib):
    assert lib.pe_workspace_bytes_filtered(0, 3) == 0 and lib.pe_workspace_bytes_filtered(-1, 3) == 0
    assert lib.pe_workspace_bytes_filtered(2, 3) > lib.pe_workspace_bytes_filtered(1, 3) > 0
    assert lib.pe_workspace_bytes_filtered(1, 256) == 0
    assert lib.pe_workspace_bytes_weigh(14, 64, 10, 16) > 0
    for bad in ((-1, 64, 10, 16), (14, 0, 10, 16), (14, 64, 0, 16), (14, 64, 10, 8), (14, 64, 1 << 28, 16)):
        assert lib.pe_workspace_bytes_weigh(*bad) == 0


def test_binding_refusals(lib):
    x = torch.zeros(6, 100, dtype=torch.bfloat16)
    i, w = torch.zeros(6, dtype=torch.int32), torch.zeros(6)
    with pytest.raises(ValueError):
        _native.draft_sample(x, w, i, i)
    with pytest.raises(ValueError):
        _native.verify_filtered(x, x, 2, i, w, w, i, i, i, i)
    cache = torch.zeros(2, 8, 1, 18 * 64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        _native.kv_weigh(x, cache, i.view(2, 3), None, i, None, w, w, i, i)
    with pytest.raises(ValueError):
        _native.kv_evict(cache, w, i.view(2, 3), i.view(2, 3), i, i, i.view(2, 1, 3), i, i)
    assert _native.new_kv_mass(torch.zeros(3, 2, 2, 1152, dtype=torch.uint8)).shape == (3, 2, 32)
