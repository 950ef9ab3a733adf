"""Host-side refusals of outputs that lie over a call's inputs: its blocks read them at any time up to the last
one's start.  Every call here is refused before CUDA is touched; fake pointers are never dereferenced."""
import pytest

from speculative_decoding_pe_gb300 import _native
from test_bounded_abi import EINVAL, EVICT, VERIFY, fill, lib  # noqa: F401

FAR = 0x10000


def apart(struct, at):
    """A pointer of its own for every field, but for those given."""
    names = [n for n, t in struct._fields_ if t is _native.P]
    return {n: at.get(n, FAR * (i + 2)) for i, n in enumerate(names)}


@pytest.mark.parametrize("at", [
    # (two requests of four bytes each)
    dict(out_lengths=FAR, lengths=FAR), dict(out_lengths=FAR, lengths=FAR + 4), dict(out_lengths=FAR + 4, lengths=FAR),
    dict(out_lengths=FAR, keep=FAR), dict(out_lengths=FAR + 4, keep=FAR), dict(out_lengths=FAR + 76, block_table=FAR),
    dict(out_lengths=FAR + 28, dst_table=FAR), dict(kept=FAR, lengths=FAR + 3196), dict(kept=FAR, keep=FAR + 3196),
    dict(kept=FAR, block_table=FAR + 64), dict(kept=FAR + 28, dst_table=FAR)])
def test_evict(lib, at):  # noqa: F811
    a = fill(_native.KvEvictArgs(), **EVICT, **apart(_native.KvEvictArgs, at))
    assert lib.pe_kv_evict(a, None) == EINVAL


@pytest.mark.parametrize("at", [
    # (two requests of three drafts each)
    dict(accept_prob=FAR, u_accept=FAR), dict(accept_prob=FAR + 20, u_accept=FAR), dict(accept_prob=FAR, u_accept=FAR + 20),
    dict(accept_prob=FAR, u_draw=FAR + 20), dict(accept_prob=FAR + 4, u_draw=FAR), dict(accepted_len=FAR, u_draw=FAR),
    dict(bonus_token=FAR, u_draw=FAR + 4), dict(accepted_len=FAR + 20, u_accept=FAR), dict(bonus_token=FAR, u_accept=FAR)])
def test_verify(lib, at):  # noqa: F811
    a = fill(_native.VerifyFilteredArgs(), **VERIFY, **apart(_native.VerifyFilteredArgs, at))
    assert lib.pe_verify_filtered(a, None) == EINVAL
