"""Sizes whose products pass 64 bits are refused.  The calls run in a child
process, which a division by zero on the host would end; their pointers are
fakes that no check dereferences."""
import json
import subprocess
import sys

import pytest

from speculative_decoding_pe_gb300 import build
from test_attn_abi import EINVAL

BIG = 2 ** 31 - 1
CALL = """
import ctypes, json, sys
sys.path.insert(0, %r)
from speculative_decoding_pe_gb300 import _native
from test_attn_abi import append_args, cached_args, prompt_args, FAKE
kind, over = json.loads(sys.argv[1])
lib = _native.load()
if kind == "read":
    a = {**dict(cache=FAKE, nb=10, bs=16, Hkv=8, D=64, slots=FAKE, n=4, k=FAKE, v=FAKE, err=FAKE), **over}
    print(lib.pe_kv_read(*a.values(), None))
else:
    a = dict(append=append_args, cached=cached_args, prompt=prompt_args)[kind](**over)
    print(getattr(lib, dict(append="pe_kv_append", cached="pe_attn_cached", prompt="pe_attn_prompt")[kind])(ctypes.byref(a), None))
"""


@pytest.mark.parametrize("kind, over", [
    # heads * block_size * D = 2^64: a divisor of zero in 64 bits
    ("append", dict(T=0, Hq=2 ** 30, Hkv=2 ** 30, D=128, block_size=2 ** 27)),
    ("read", dict(n=0, Hkv=2 ** 30, D=128, bs=2 ** 27)),
    ("cached", dict(T=1, Hq=2 ** 30, Hkv=2 ** 30, D=128, block_size=2 ** 27, bt_width=1)),
    # ... = 2^63: negative
    ("append", dict(T=0, Hq=2 ** 29, Hkv=2 ** 29, D=128, block_size=2 ** 27)),
    # T (Hq + 2 Hkv) past 2^63
    ("append", dict(T=BIG, Hq=BIG, Hkv=BIG)),
    # T Hq D = 2^66, and one that wraps to a negative number
    ("cached", dict(T=2 ** 30, Hq=2 ** 30, Hkv=2 ** 23, D=64)),
    ("cached", dict(T=BIG, Hq=BIG, Hkv=BIG, D=64)),
    ("prompt", dict(T=2 ** 30, Hq=2 ** 30, Hkv=2 ** 23, D=64)),
    ("prompt", dict(T=BIG, Hq=BIG, Hkv=BIG, D=128))])
def test_sizes_past_64_bits(kind, over):
    build.build()
    r = subprocess.run([sys.executable, "-c", CALL % __file__.rsplit("/", 1)[0], json.dumps([kind, over])],
                       capture_output=True, text=True, cwd=build.ROOT)
    assert r.returncode == 0, "%s ended by %d" % (kind, r.returncode)
    assert int(r.stdout) == EINVAL
